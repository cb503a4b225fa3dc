"""What is measured of the operators of a hybrid stack's decode step, and their plain forms.

  pool    kda_decode_pool: the gated delta rule's recurrent form over a pool of states
  append  kda_kv_append: new keys and values into a paged cache, rotary rotation on the way
  attend  kda_kv_decode: softmax attention of the newest tokens over the paged cache

`own` False runs the plain forms (elementary torch operations in 32 bits), True the library.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f32": 4, "e4m3": 1}


def listed():
    return [
        # --- pool: N sequences, `new_lo`..`new_hi` tokens each.
        # A handful of sequences of a small stack: the latency of one step.
        dict(name="pool 4x1 h8", op="pool", N=4, Hk=8, Hv=8, D=128, dtype="bf16", new_lo=1, new_hi=1, keep="last",
             gate="channel", raw=False, seed=1),
        # Full batch decode, one token a sequence, in place in the pool (the decode benchmark's sizes).
        dict(name="pool 256x1 h32", op="pool", N=256, Hk=32, Hv=32, D=128, dtype="bf16", new_lo=1, new_hi=1,
             keep="last", gate="channel", raw=False, seed=2),
        # Verification of drafts: every token's state kept for the roll back, shared q/k heads, a scalar
        # gate, raw projections (logits, q and k not normalised).
        dict(name="pool drafts h16/32", op="pool", N=64, Hk=16, Hv=32, D=128, dtype="bf16", new_lo=1, new_hi=5,
             keep="all", gate="scalar", raw=True, seed=3),
        # Short catch-up of several tokens, fp32 with the smaller head.
        dict(name="pool f32 d64 catch-up", op="pool", N=33, Hk=12, Hv=12, D=64, dtype="f32", new_lo=1, new_hi=16,
             keep="last", gate="channel", raw=False, seed=4),
        # --- append: the new tokens' q, k, v are slices of one fused projection.
        # One token for each of 64 sequences.
        dict(name="append 64x1", op="append", N=64, new_lo=1, new_hi=1, past=8192, Hq=32, Hkv=8, D=128,
             dtype="bf16", cache="bf16", page=16, rot=128, axes=1, adjacent=False, seed=5),
        # Prompts of a ragged batch.
        dict(name="append prompts", op="append", N=6, new_lo=1024, new_hi=8192, past=2048, Hq=32, Hkv=8, D=128,
             dtype="bf16", cache="bf16", page=64, rot=128, axes=1, adjacent=False, seed=6),
        # Image and video tokens: positions in time, height and width, half of the channels rotated, 8-bit cache.
        dict(name="append video e4m3", op="append", N=3, new_lo=700, new_hi=5000, past=500, Hq=16, Hkv=4, D=128,
             dtype="bf16", cache="e4m3", page=32, rot=64, axes=3, adjacent=True, seed=7),
        # --- attend: `len_lo`..`len_hi` keys a sequence, the newest `new_lo`..`new_hi` of them with queries.
        # A few short chats: latency.
        dict(name="attend 8 short", op="attend", N=8, new_lo=1, new_hi=1, len_lo=1, len_hi=300, Hq=32, Hkv=8, D=128,
             dtype="bf16", cache="bf16", page=16, cap=0.0, window=0, bias=False, start=False, seed=8),
        # A serving batch with lengths that differ by a factor of 32.
        dict(name="attend 64 ragged", op="attend", N=64, new_lo=1, new_hi=1, len_lo=512, len_hi=16384, Hq=32, Hkv=8,
             D=128, dtype="bf16", cache="bf16", page=64, cap=0.0, window=0, bias=False, start=False, seed=9),
        # One request with a long context.
        dict(name="attend 1 long", op="attend", N=1, new_lo=1, new_hi=1, len_lo=262143, len_hi=262143, Hq=64, Hkv=8,
             D=128, dtype="bf16", cache="bf16", page=64, cap=0.0, window=0, bias=False, start=False, seed=10),
        # Drafts over an 8-bit cache, capped scores, a sliding window, an odd group of heads.
        dict(name="attend drafts e4m3", op="attend", N=48, new_lo=2, new_hi=6, len_lo=64, len_hi=16384, Hq=40, Hkv=8,
             D=128, dtype="bf16", cache="e4m3", page=128, cap=30.0, window=4096, bias=False, start=False, seed=11),
        # fp32, one query head a key head, a bias by distance, document starts.
        dict(name="attend f32 d64 bias", op="attend", N=16, new_lo=1, new_hi=1, len_lo=100, len_hi=4096, Hq=12, Hkv=12,
             D=64, dtype="f32", cache="f32", page=16, cap=0.0, window=0, bias=True, start=True, seed=12),
    ]


def draw(rng):
    def log(lo, hi):
        return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))

    op = rng.choice(["pool", "append", "attend"])
    D = rng.choice([64, 128])
    seed = rng.randrange(100, 1 << 30)
    if op == "pool":
        group = rng.choice([1, 1, 2, 4])
        Hk = log(1, 32 // group)
        new_hi = rng.choice([1, 1, 2, 3, 4, 6, 8, 16])
        new_lo = rng.randint(1, new_hi)
        keep = rng.choice(["last", "all"])
        states = 8192 * 128 * 128 // (D * D) // ((1 + new_hi) if keep == "all" else max(1, new_hi // 2))
        return dict(op=op, N=log(1, max(1, min(256, states // (Hk * group)))), Hk=Hk, Hv=Hk * group, D=D,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), new_lo=new_lo, new_hi=new_hi, keep=keep,
                    gate=rng.choice(["channel", "scalar"]), raw=rng.choice([False, True]), seed=seed)
    Hkv = log(1, 16)
    Hq = Hkv * rng.choice([1, 2, 4, 5, 7, 8])
    dtype, cache = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("bf16", "e4m3"), ("f32", "f32")])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        tokens = log(1, min(32768, (1 << 27) // ((Hq + 2 * Hkv) * D)))
        N = log(1, min(tokens, 256))
        mean = tokens // N
        return dict(op=op, N=N, new_lo=max(1, mean // 2), new_hi=mean, past=log(1, 8192), Hq=Hq, Hkv=Hkv, D=D,
                    dtype=dtype, cache=cache, page=page, rot=rng.choice([D, D, D // 2, 32]), axes=rng.choice([1, 1, 3]),
                    adjacent=rng.choice([False, True]), seed=seed)
    N = log(1, 128)
    len_hi = log(1, max(1, min(131072, (1 << 29) // (Hkv * D * BYTES[cache] * N))))
    new_hi = min(len_hi, rng.choice([1, 1, 1, 2, 3, 5, 8]))
    return dict(op=op, N=N, new_lo=rng.randint(1, new_hi), new_hi=new_hi, len_lo=max(new_hi, len_hi // 16), len_hi=len_hi,
                Hq=Hq, Hkv=Hkv, D=D, dtype=dtype, cache=cache, page=page, cap=rng.choice([0.0, 0.0, 20.0, 50.0]),
                window=rng.choice([0, 0, 128, 1000, 4096]), bias=rng.choice([False, False, True]),
                start=rng.choice([False, False, True]), seed=seed)


def _new(case):
    """New tokens of each sequence: by the case alone, so that work() knows them."""
    r = random.Random(case["seed"])
    return [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["N"])]


def _past(case):
    """Keys that each sequence holds after the call."""
    r = random.Random(case["seed"] + 1)
    new = _new(case)
    if case["op"] == "append":
        return [n + r.randint(case["past"] // 2, case["past"]) for n in new]
    lo, hi = math.log(case["len_lo"]), math.log(case["len_hi"] + 1)
    return [max(n, min(case["len_hi"], int(math.exp(r.uniform(lo, hi))))) for n in new]


def _starts(case):
    """First visible key of each sequence (the start of its last document)."""
    r = random.Random(case["seed"] + 2)
    return [r.randint(0, (n - 1) // 4) if case.get("start") else 0 for n in _past(case)]


def _axis_pairs(case):
    pairs, axes = case["rot"] // 2, case["axes"]
    if axes == 1:
        return [pairs]
    per = pairs * 3 // 8
    return [pairs - 2 * per, per, per]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed * 1000003 + case["seed"])

    def randn(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32).to(dtype)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device=dev)

    N, D, new = case["N"], case["D"], _new(case)
    T = sum(new)
    dt = DTYPES[case["dtype"]]
    cu = ints([sum(new[:n]) for n in range(N + 1)])
    s = dict(case=case, new=new, cu=None if max(new) == min(new) == 1 else cu)
    # where each packed token stands: its sequence and its place in it
    s["seq"] = torch.repeat_interleave(torch.arange(N, device=dev), ints(new).long())
    s["place"] = torch.arange(T, device=dev) - cu[:-1].long()[s["seq"]]
    if case["op"] == "pool":
        Hk, Hv = case["Hk"], case["Hv"]
        qkv = randn(T, (2 * Hk + Hv) * D)
        q, k = qkv[:, : Hk * D].view(T, Hk, D), qkv[:, Hk * D : 2 * Hk * D].view(T, Hk, D)
        if not case["raw"]:
            q /= q.norm(dim=-1, keepdim=True)
            k /= k.norm(dim=-1, keepdim=True)
        qkv = qkv.to(dt)  # q, k and v: slices of one projection
        s["q"], s["k"] = qkv[:, : Hk * D].view(T, Hk, D), qkv[:, Hk * D : 2 * Hk * D].view(T, Hk, D)
        s["v"] = qkv[:, 2 * Hk * D :].view(T, Hv, D)
        g = 3.0 + randn(*((T, Hv) if case["gate"] == "scalar" else (T, Hv, D)))
        b = randn(T, Hv)
        s["g"] = g if case["raw"] else torch.nn.functional.logsigmoid(g)
        s["beta"] = b if case["raw"] else torch.sigmoid(b)
        kept = N if case["keep"] == "last" else N + T
        spare = 1 + kept // 16
        s["pool"] = randn(kept + spare, Hv, D, D) * 0.02
        slots = torch.randperm(kept + spare, generator=gen, device=dev)[:kept].to(torch.int32)
        s["slots_in"] = slots[:N].contiguous()
        if case["keep"] == "last":  # in place, after the last token only
            s["slots_out"] = torch.full((T,), -1, dtype=torch.int32, device=dev)
            s["slots_out"][cu[1:].long() - 1] = s["slots_in"]
        else:  # a slot for every token; the state before the draft stays
            s["slots_out"] = slots[N:].contiguous()
        s["out"] = torch.empty(T, Hv, D, dtype=dt, device=dev)
        return s
    Hq, Hkv, ps, lens = case["Hq"], case["Hkv"], case["page"], _past(case)
    s["lens"] = ints(lens)
    pages = [-(-n // ps) for n in lens]
    total = sum(pages) + 2
    order = torch.randperm(total, generator=gen, device=dev).to(torch.int32)
    table = torch.full((N, max(pages)), -1, dtype=torch.int32, device=dev)
    at = 0
    for n in range(N):
        table[n, : pages[n]] = order[at : at + pages[n]]
        at += pages[n]
    s["table"] = table
    cdt = DTYPES[case["cache"]]
    s["ks"] = s["vs"] = None
    if case["cache"] == "e4m3":
        s["ks"] = 0.01 + 0.01 * torch.rand(Hkv, generator=gen, device=dev)
        s["vs"] = 0.01 + 0.01 * torch.rand(Hkv, generator=gen, device=dev)

    def cache(scale):
        c = torch.empty(total, Hkv, ps, D, dtype=cdt, device=dev)
        for i in range(0, total, 1024):  # in pieces: the float32 draw of a large cache is larger still
            x = randn(min(1024, total - i), Hkv, ps, D)
            c[i : i + 1024] = (x if scale is None else (x / scale[:, None, None]).clamp(-448, 448)).to(cdt)
        return c

    s["kc"], s["vc"] = cache(s["ks"]), cache(s["vs"])
    if case["op"] == "append":
        qkv = randn(T, (Hq + 2 * Hkv) * D, dtype=dt)
        s["q"] = qkv[:, : Hq * D].view(T, Hq, D)
        s["k"] = qkv[:, Hq * D : (Hq + Hkv) * D].view(T, Hkv, D)
        s["v"] = qkv[:, (Hq + Hkv) * D :].view(T, Hkv, D)
        s["q_out"] = torch.empty(T, Hq, D, dtype=dt, device=dev)
        half = case["rot"] // 2
        s["inv_freq"] = (10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)).float().to(dev)
        s["pairs"] = _axis_pairs(case)
        s["positions"] = None
        if case["axes"] > 1:  # time, height, width
            s["positions"] = torch.stack([torch.randint(0, m, (T,), generator=gen, device=dev, dtype=torch.int32)
                                          for m in (100000, 64, 96)]).contiguous()
        return s
    s["q"] = randn(T, Hq, D, dtype=dt)
    s["out"] = torch.empty(T, Hq, D, dtype=dt, device=dev)
    s["lse"] = torch.empty(T, Hq, dtype=torch.float32, device=dev)
    s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, Hq + 1, device=dev, dtype=torch.float32) / Hq) if case["bias"] else None
    s["start"] = ints(_starts(case)) if case["start"] else None
    s["scale"] = D ** -0.5
    s["max_q"] = max(new)
    s["workspace"] = torch.empty(64 << 20, dtype=torch.uint8, device=dev)  # a serving program keeps one for all its layers
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        from linear_attention_rule_b200 import kda

        if op == "pool":
            flags = kda.KDA_IN_G_SCALAR if s["case"]["gate"] == "scalar" else 0
            if s["case"]["raw"]:
                flags |= kda.KDA_IN_NORMALIZE_QK | kda.KDA_IN_G_LOGITS | kda.KDA_IN_BETA_LOGITS
            kda.kda_decode_pool(s["q"], s["k"], s["v"], s["g"], s["beta"], s["pool"], s["slots_in"], s["slots_out"],
                                s["out"], cu_seqlens=s["cu"], in_flags=flags)
            return {"out": s["out"], "pool": s["pool"]}
        if op == "append":
            kda.kda_kv_append(s["k"], s["v"], s["kc"], s["vc"], s["table"], s["lens"], cu_seqlens=s["cu"], q=s["q"],
                              q_out=s["q_out"], inv_freq=s["inv_freq"], positions=s["positions"],
                              axis_pairs=s["pairs"], adjacent=s["case"]["adjacent"], k_scale=s["ks"], v_scale=s["vs"])
            return {"q": s["q_out"], "k_cache": s["kc"], "v_cache": s["vc"]}
        kda.kda_kv_decode(s["q"], s["kc"], s["vc"], s["table"], s["lens"], s["out"], cu_seqlens=s["cu"],
                          max_q=s["max_q"], scale=s["scale"], softcap=s["case"]["cap"], window=s["case"]["window"],
                          alibi_slopes=s["slopes"], kv_start=s["start"], lse=s["lse"], k_scale=s["ks"],
                          v_scale=s["vs"], workspace=s["workspace"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "pool":
        return _plain_pool(s)
    if op == "append":
        return _plain_append(s)
    return _plain_attend(s)


def _padded(s, x):
    """Packed tokens [T, ...] as [N, longest, ...], zeros behind the short ones."""
    y = x.new_zeros((s["case"]["N"], max(s["new"])) + tuple(x.shape[1:]))
    y[s["seq"], s["place"]] = x
    return y


def _plain_pool(s):
    c = s["case"]
    q, k, v, g, b = (s[n].float() for n in ("q", "k", "v", "g", "beta"))
    if c["raw"]:
        q = q / q.square().sum(-1, keepdim=True).sqrt().clamp_min(1e-12)
        k = k / k.square().sum(-1, keepdim=True).sqrt().clamp_min(1e-12)
        a, b = torch.sigmoid(g), torch.sigmoid(b)
    else:
        a = torch.exp(g)
    if c["gate"] == "scalar":
        a = a[..., None]
    group = c["Hv"] // c["Hk"]
    q, k = q.repeat_interleave(group, 1), k.repeat_interleave(group, 1)
    q, k, v, a, b, to = (_padded(s, x) for x in (q, k, v, a, b, s["slots_out"] + 1))
    there = _padded(s, torch.ones_like(s["slots_out"]))
    S = s["pool"][s["slots_in"].long()]
    o = torch.zeros_like(v)
    for t in range(max(s["new"])):  # the recurrence over the tokens
        S = S * a[:, t, :, :, None]
        u = b[:, t, :, None] * (v[:, t] - (S * k[:, t, :, :, None]).sum(2))
        S = S + k[:, t, :, :, None] * u[:, :, None, :]
        o[:, t] = (S * q[:, t, :, :, None]).sum(2)
        keep = (there[:, t] > 0) & (to[:, t] > 0)
        s["pool"][to[keep, t].long() - 1] = S[keep]
    s["out"].copy_(o[s["seq"], s["place"]])
    return {"out": s["out"], "pool": s["pool"]}


def _rotate(x, cos, sin, adjacent):
    """x [T, H, D] with its first 2 * pairs channels rotated by the angles [T, pairs]."""
    rot, c, d = 2 * cos.shape[1], cos[:, None, :], sin[:, None, :]
    y = x.clone()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if adjacent else (x[..., : rot // 2], x[..., rot // 2 : rot])
    if adjacent:
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * d, b * c + a * d
    else:
        y[..., : rot // 2], y[..., rot // 2 : rot] = a * c - b * d, b * c + a * d
    return y


def _plain_append(s):
    c = s["case"]
    new = torch.bincount(s["seq"], minlength=c["N"])
    at = s["lens"].long()[s["seq"]] - new[s["seq"]] + s["place"]  # place in the sequence, and so in the cache
    if s["positions"] is None:
        angle = at.double()[:, None] * s["inv_freq"].double()
    else:
        axis = torch.repeat_interleave(torch.arange(c["axes"], device=at.device), torch.tensor(s["pairs"], device=at.device))
        angle = s["positions"].double()[axis].t() * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    s["q_out"].copy_(_rotate(s["q"].float(), cos, sin, c["adjacent"]))
    k, v = _rotate(s["k"].float(), cos, sin, c["adjacent"]), s["v"].float()
    page, row = s["table"][s["seq"], at // c["page"]].long(), at % c["page"]
    if c["cache"] == "e4m3":
        k = (k / s["ks"][:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        v = (v / s["vs"][:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        s["kc"].view(torch.uint8)[page, :, row] = k.view(torch.uint8)
        s["vc"].view(torch.uint8)[page, :, row] = v.view(torch.uint8)
    else:
        s["kc"][page, :, row] = k.to(s["kc"].dtype)
        s["vc"][page, :, row] = v.to(s["vc"].dtype)
    return {"q": s["q_out"], "k_cache": s["kc"], "v_cache": s["vc"]}


def _plain_attend(s):
    c = s["case"]
    N, D, Hkv, G = c["N"], c["D"], c["Hkv"], c["Hq"] // c["Hkv"]
    q = _padded(s, s["q"].float())  # [N, Tq, Hq, D]
    Tq = q.shape[1]
    q = q.view(N, Tq, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(N, Hkv, Tq * G, D)
    pages = s["table"].long().clamp_min(0)
    L = pages.shape[1] * c["page"]
    k = s["kc"][pages].permute(0, 2, 1, 3, 4).reshape(N, Hkv, L, D).float()
    v = s["vc"][pages].permute(0, 2, 1, 3, 4).reshape(N, Hkv, L, D).float()
    if s["ks"] is not None:
        k, v = k * s["ks"][:, None, None], v * s["vs"][:, None, None]
    x = torch.matmul(q, k.transpose(2, 3)).view(N, Hkv, Tq, G, L) * s["scale"]
    if c["cap"]:
        x = c["cap"] * torch.tanh(x / c["cap"])
    new = torch.bincount(s["seq"], minlength=N)
    i = (s["lens"].long() - new)[:, None] + torch.arange(Tq, device=q.device)  # [N, Tq]
    j = torch.arange(L, device=q.device)
    gap = (j - i[:, :, None])[:, None, :, None, :]
    if c["bias"]:
        x = x + s["slopes"].view(1, Hkv, 1, G, 1) * gap
    seen = gap <= 0
    if c["window"]:
        seen = seen & (gap > -c["window"])
    if c["start"]:
        seen = seen & (j >= s["start"].long()[:, None])[:, None, None, None, :]
    x = torch.where(seen, x, float("-inf"))
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - top)
    den = p.sum(-1, keepdim=True)
    o = torch.matmul((p / den).view(N, Hkv, Tq * G, L), v)
    o = o.view(N, Hkv, Tq, G, D).permute(0, 2, 1, 3, 4).reshape(N, Tq, c["Hq"], D)
    lse = (top + torch.log(den)).squeeze(-1).permute(0, 2, 1, 3).reshape(N, Tq, c["Hq"])
    s["out"].copy_(o[s["seq"], s["place"]])
    s["lse"].copy_(lse[s["seq"], s["place"]])
    return {"out": s["out"], "lse": s["lse"]}


def work(case):
    new = _new(case)
    N, T, D, e = case["N"], sum(new), case["D"], BYTES[case["dtype"]]
    if case["op"] == "pool":
        state = case["Hv"] * D * D * 4
        kept = N if case["keep"] == "last" else T
        gates = T * case["Hv"] * 4 * (1 + (1 if case["gate"] == "scalar" else D))
        return {"bytes": (N + kept) * state + T * (2 * case["Hk"] + 2 * case["Hv"]) * D * e + gates,
                "flops": 7.0 * T * case["Hv"] * D * D}
    Hq, Hkv, ce = case["Hq"], case["Hkv"], BYTES[case["cache"]]
    if case["op"] == "append":
        return {"bytes": T * D * (2 * Hq * e + 2 * Hkv * (e + ce)), "flops": 3.0 * T * (Hq + Hkv) * case["rot"]}
    keys = pairs = 0
    for n, length, start in zip(new, _past(case), _starts(case)):
        first = max(start, length - n - case["window"] + 1 if case["window"] else 0)
        keys += length - first
        for t in range(length - n, length):
            pairs += t + 1 - max(start, t - case["window"] + 1 if case["window"] else 0)
    return {"bytes": 2.0 * keys * Hkv * D * ce + 2 * T * Hq * D * e + 4 * T * Hq, "flops": 4.0 * pairs * Hq * D}


def exact(case, seed):
    """The definitions in 64 bits, sequence by sequence."""
    s = prepare(case, seed)
    N, D, new = case["N"], case["D"], s["new"]
    first = [sum(new[:n]) for n in range(N)]
    if case["op"] == "pool":
        Hk, Hv = case["Hk"], case["Hv"]
        if N * Hv * D * D > 1 << 28:
            return None
        out = torch.zeros(sum(new), Hv, D, dtype=torch.float64, device="cuda")
        pool = s["pool"].double()
        head = torch.arange(Hv, device="cuda") // (Hv // Hk)
        for n in range(N):
            S = pool[int(s["slots_in"][n])].clone()
            for t in range(first[n], first[n] + new[n]):
                q, k, v = s["q"][t].double()[head], s["k"][t].double()[head], s["v"][t].double()
                g, b = s["g"][t].double(), s["beta"][t].double()
                if case["raw"]:
                    q, k = (x / torch.linalg.vector_norm(x, dim=-1, keepdim=True) for x in (q, k))
                    g, b = -torch.log1p(torch.exp(-g)), 1 / (1 + torch.exp(-b))
                S = torch.exp(g).reshape(Hv, -1, 1) * S
                read = torch.bmm(k[:, None, :], S)[:, 0]
                S = S + torch.bmm(k[:, :, None], (b[:, None] * (v - read))[:, None, :])
                out[t] = torch.bmm(q[:, None, :], S)[:, 0]
                if int(s["slots_out"][t]) >= 0:
                    pool[int(s["slots_out"][t])] = S
        return {"out": out, "pool": pool}
    if case["op"] == "append":
        turned = []
        lens, cu = s["lens"].tolist(), first
        at = torch.cat([torch.arange(lens[n] - new[n], lens[n], device="cuda") for n in range(N)])
        pos = at[None].expand(case["axes"], -1) if s["positions"] is None else s["positions"]
        freq = s["inv_freq"].double()
        unit, k0 = [], 0
        for a, m in enumerate(s["pairs"]):
            unit.append(torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), pos[a].double()[:, None] * freq[None, k0 : k0 + m]))
            k0 += m
        unit = torch.cat(unit, 1)[:, None, :]
        for x in (s["q"].double(), s["k"].double()):
            r = x[..., : case["rot"]]
            if case["adjacent"]:
                z = torch.view_as_complex(r.reshape(*r.shape[:2], -1, 2).contiguous()) * unit
                r = torch.view_as_real(z).reshape(r.shape)
            else:
                h = case["rot"] // 2
                z = torch.complex(r[..., :h].contiguous(), r[..., h:].contiguous()) * unit
                r = torch.cat([z.real, z.imag], -1)
            turned.append(torch.cat([r, x[..., case["rot"] :]], -1))
        caches = []
        for x, c, scale in ((turned[1], s["kc"], s["ks"]), (s["v"].double(), s["vc"], s["vs"])):
            c = c.double()
            if scale is not None:
                x = (x / scale.double()[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).double()
            for n in range(N):
                rows = torch.arange(lens[n] - new[n], lens[n], device="cuda")
                where = s["table"][n].long()[rows // case["page"]]
                c[where, :, rows % case["page"]] = x[cu[n] : cu[n] + new[n]]
            caches.append(c)
        return {"q": turned[0], "k_cache": caches[0], "v_cache": caches[1]}
    Hq, Hkv, ps = case["Hq"], case["Hkv"], case["page"]
    out = torch.zeros(sum(new), Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(sum(new), Hq, dtype=torch.float64, device="cuda")
    lens, starts, total = s["lens"].tolist(), _starts(case), 0
    for n in range(N):
        total += lens[n] * Hkv * D
    if total > 1 << 31:
        return None
    for n in range(N):
        ids = s["table"][n, : -(-lens[n] // ps)].long()
        K, V = (c[ids].double().transpose(0, 1).reshape(Hkv, -1, D)[:, : lens[n]] for c in (s["kc"], s["vc"]))
        if s["ks"] is not None:
            K, V = K * s["ks"].double()[:, None, None], V * s["vs"].double()[:, None, None]
        for t in range(new[n]):
            i = lens[n] - new[n] + t
            lo = max(starts[n], i - case["window"] + 1 if case["window"] else 0)
            q = s["q"][first[n] + t].double().view(Hkv, Hq // Hkv, D)
            x = torch.bmm(q, K[:, lo : i + 1].transpose(1, 2)) / math.sqrt(D)
            if case["cap"]:
                x = torch.tanh(x / case["cap"]) * case["cap"]
            if case["bias"]:
                back = torch.arange(lo - i, 1, device="cuda", dtype=torch.float64)
                x = x + s["slopes"].double().view(Hkv, -1, 1) * back
            out[first[n] + t] = torch.bmm(torch.softmax(x, -1), V[:, lo : i + 1]).reshape(Hq, D)
            lse[first[n] + t] = torch.logsumexp(x, -1).reshape(Hq)
    return {"out": out, "lse": lse}
