"""Operators that stand between the 4-bit linears of a transformer block.

Three families, each in a plain form (elementary torch operations in 32 bits,
64 where a rounding border needs it) and as calls of the library:

  norm     residual_norm: post-norm, gate and residual scale, pre-norm with
           modulation, in one pass over the rows
  lora     lora_linear: low-rank adapters of many requests beside a shared
           projection
  cache    kv4_append + kv4_read: keys and values through the 4-bit cache
  attend   kv4_attention: attention of new rows over that cache

`own` selects which one `run` computes.  Nothing outside a case and a seed
enters: the case fixes the sizes, lengths and assignments, the seed the values.
"""
import math
import random

import torch

own = False

DEV = "cuda"
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def _lib():
    import w4a4_rank_corrected_quantize_amd as svdq
    return svdq


# ------------------------------------------------------------------- cases

def _norm(name, M, D, post="none", pre="rms", affine=False, gate=True, mod=True, images=1, ragged=False, fp32=False,
          alpha=1.0, shape_seed=0):
    return dict(name=name, op="norm", M=M, D=D, post=post, pre=pre, affine=affine, gate=gate, mod=mod, images=images,
                ragged=ragged, fp32=fp32, alpha=alpha, shape_seed=shape_seed)


def _lora(name, M, K, N, R, adapters, runs, none=0.0, shape_seed=0):
    return dict(name=name, op="lora", M=M, K=K, N=N, R=R, adapters=adapters, runs=runs, none=none,
                shape_seed=shape_seed)


def _cache(name, prec, T, heads, dim, page, shape_seed=0):
    return dict(name=name, op="cache", prec=prec, T=T, heads=heads, dim=dim, page=page, shape_seed=shape_seed)


def _attend(name, prec, B, heads_q, heads_kv, dim, page, q_max, kv_max, q_min=1, kv_min=1, causal=True, window=0,
            shape_seed=0):
    return dict(name=name, op="attend", prec=prec, B=B, heads_q=heads_q, heads_kv=heads_kv, dim=dim, page=page,
                q_min=q_min, q_max=q_max, kv_min=kv_min, kv_max=kv_max, causal=causal, window=window,
                shape_seed=shape_seed)


def listed():
    return [
        # one token of a decoder between attention and MLP: latency
        _norm("norm_token", 1, 4096, pre="rms", affine=True, gate=False, mod=False),
        # a 1024 x 1024 image (4096 patches + 512 text tokens) times two prompts, LayerNorm without weights and the
        # modulation vectors of the AWQ layer
        _norm("norm_images", 9216, 4096, pre="layer", images=2),
        # packed requests of different lengths, norms on both sides of the block, stream held in fp32
        _norm("norm_packed_fp32", 1337, 2560, post="rms", pre="rms", affine=True, images=7, ragged=True, fp32=True,
              alpha=0.5, shape_seed=3),
        # decoding: every row its own adapter
        _lora("lora_decode", 16, 4096, 4096, 16, 16, 16),
        # a mixed step: short runs of seven adapters, some rows without one
        _lora("lora_mixed", 1111, 2048, 6144, 32, 7, 29, none=0.25, shape_seed=5),
        # two images with an adapter each through the MLP's first linear
        _lora("lora_images", 9216, 4096, 12288, 64, 2, 2),
        # the text tokens of two prompts enter the cache
        _cache("cache_text", "mxfp4", 1024, 24, 128, 64, shape_seed=2),
        # all tokens of an image, heads of 64
        _cache("cache_image", "int4", 4608, 32, 64, 128),
        # one short request decodes a token
        _attend("attend_token", "int4", 1, 32, 8, 128, 16, 1, 1000, kv_min=1000),
        # a batch of long requests decodes a token each
        _attend("attend_decode", "mxfp4", 32, 32, 8, 128, 64, 1, 16384, kv_min=4097, shape_seed=7),
        # mixed step: prompts in chunks beside single tokens
        _attend("attend_chunks", "int4", 8, 16, 4, 64, 32, 700, 6000, shape_seed=11),
        # image tokens over the cached tokens of image and text, every head its own keys
        _attend("attend_image", "mxfp4", 1, 24, 24, 128, 64, 4608, 4608, q_min=4608, kv_min=4608, causal=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "lora", "cache", "attend"])
    s = rng.randrange(1 << 30)
    if op == "norm":
        D = 8 * _log_int(rng, 8, 1024)
        M = _log_int(rng, 1, max(1, min(20000, 9216 * 4096 // D)))
        mod = rng.random() < 0.7
        return _norm("", M, D, post=rng.choice(["none", "rms", "layer"]), pre=rng.choice(["rms", "layer"]),
                     affine=rng.random() < 0.5, gate=rng.random() < 0.7, mod=mod, images=rng.randint(1, min(M, 12)),
                     ragged=True, fp32=rng.random() < 0.4, alpha=rng.choice([1.0, 0.5, 0.125]), shape_seed=s)
    if op == "lora":
        K = 8 * _log_int(rng, 32, 1024)
        N = 8 * _log_int(rng, 32, 1024)
        M = _log_int(rng, 1, min(9216, 9216 * 16384 // (K + N)))
        n = _log_int(rng, 1, 32)
        return _lora("", M, K, N, 8 * rng.randint(1, 8), n, rng.randint(1, 2 * n), none=rng.choice([0.0, 0.25]),
                     shape_seed=s)
    if op == "cache":
        heads, dim = rng.randint(1, 32), rng.choice([64, 128])
        return _cache("", rng.choice(["int4", "mxfp4"]), _log_int(rng, 1, 4608 * 32 * 64 // (heads * dim)), heads, dim,
                      rng.choice([16, 32, 64, 128]), shape_seed=s)
    dim, hkv = rng.choice([64, 128]), rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 8])
    q_max = 1 if rng.random() < 0.5 else _log_int(rng, 2, 1200)
    B = _log_int(rng, 1, 32 if q_max == 1 else 8)
    kv_max = max(q_max, _log_int(rng, 1, 12000 if q_max == 1 else 5000))
    if q_max > 1:       # no more products than the largest listed case
        kv_max = max(q_max, min(kv_max, int(2.5e11 / (4 * dim * hq * B * q_max))))
    causal = rng.random() < 0.7
    return _attend("", rng.choice(["int4", "mxfp4"]), B, hq, hkv, dim, rng.choice([16, 32, 64, 128]), q_max, kv_max,
                   causal=causal, window=rng.choice([0, 0, 513]) if causal else 0, shape_seed=s)


# --------------------------------------------- sizes that a case stands for

def _cuts(rng, total, parts):
    """total split into `parts` runs of at least one."""
    parts = max(1, min(parts, total))
    at = sorted(rng.sample(range(1, total), parts - 1)) if parts > 1 else []
    at = [0] + at + [total]
    return [b - a for a, b in zip(at, at[1:])]


def _norm_rows(case):
    """Modulation row of every token."""
    rng = random.Random(case["shape_seed"])
    M, B = case["M"], case["images"]
    runs = _cuts(rng, M, B) if case["ragged"] else [M // B] * B
    return [b for b, n in enumerate(runs) for _ in range(n)]


def _lora_rows(case):
    """Adapter of every row, -1 for none; consecutive runs, as requests are laid out."""
    rng = random.Random(case["shape_seed"])
    out, n = [], case["adapters"]
    for i, length in enumerate(_cuts(rng, case["M"], case["runs"])):
        a = -1 if rng.random() < case["none"] else (i if i < n else rng.randrange(n))
        out += [a] * length
    return out


def _slots(case):
    """Slots of the tokens: pages in a shuffled order; and the number of pages."""
    rng = random.Random(case["shape_seed"])
    P = case["page"]
    pages = -(-case["T"] // P) + 3
    order = list(range(pages))
    rng.shuffle(order)
    return [order[t // P] * P + t % P for t in range(case["T"])], pages


def _lengths(case):
    """(queries, keys) of every sequence; keys >= queries."""
    rng = random.Random(case["shape_seed"])
    out = []
    for _ in range(case["B"]):
        q = rng.randint(case["q_min"], case["q_max"])
        if case["q_min"] == 1 and case["q_max"] > 1 and rng.random() < 0.4:
            q = 1
        kv = max(q, rng.randint(case["kv_min"], case["kv_max"]))
        out.append((q, kv))
    return out


def _tables(case):
    rng = random.Random(case["shape_seed"] + 1)
    P = case["page"]
    need = [-(-kv // P) for _, kv in _lengths(case)]
    pages = sum(need) + 1
    order = list(range(pages))
    rng.shuffle(order)
    width = max(need)
    tables, at = [], 0
    for n in need:
        tables.append(order[at:at + n] + [0] * (width - n))
        at += n
    return tables, pages


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, scale=1.0, dtype=BF):
    return (torch.randn(*shape, generator=g, device=DEV, dtype=F32) * scale).to(dtype)


def _activations(g, *shape):
    """Normal values with a few strong channels, as activations have."""
    x = torch.randn(*shape, generator=g, device=DEV, dtype=F32)
    hot = torch.randint(0, shape[-1], (max(1, shape[-1] // 64),), generator=g, device=DEV)
    x[..., hot] *= 8.0
    return x.to(BF)


def _int(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device=DEV)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    if case["op"] == "norm":
        M, D, B = case["M"], case["D"], case["images"]
        s["r"] = _activations(g, M, D).to(F32 if case["fp32"] else BF)
        s["y"] = _activations(g, M, D)
        mods = _randn(g, B, 3 * D, scale=0.5)        # shift, scale, gate as one layer writes them
        s["shift"], s["scale"], s["gate"] = mods[:, :D], mods[:, D:2 * D], mods[:, 2 * D:]
        s["w"] = (1.0 + 0.2 * torch.randn(D, generator=g, device=DEV)).to(BF) if case["affine"] else None
        s["b"] = _randn(g, D, scale=0.1) if case["affine"] and case["pre"] == "layer" else None
        s["pw"] = (1.0 + 0.2 * torch.randn(D, generator=g, device=DEV)).to(BF) if case["affine"] else None
        s["index"] = _int(_norm_rows(case))
        if not case["gate"]:
            s["gate"] = None
        if not case["mod"]:
            s["shift"] = s["scale"] = None
    elif case["op"] == "lora":
        M, K, N, R, n = (case[k] for k in ("M", "K", "N", "R", "adapters"))
        s["X"] = _activations(g, M, K)
        s["A"] = _randn(g, n, R, K, scale=K ** -0.5)
        s["B"] = _randn(g, n, N, R, scale=R ** -0.5)
        s["scale"] = 0.25 + torch.rand(n, generator=g, device=DEV)
        s["base"] = _randn(g, M, N)
        rows = _lora_rows(case)
        s["index"] = _int(rows)
        if own:
            svdq = _lib()
            s["plan"] = svdq.lora_plan(s["index"], n)
            s["Y"] = torch.empty_like(s["base"])
            s["work"] = svdq.lora_workspace(M, K, R, n)
        else:
            s["groups"] = [(a, _int([m for m, v in enumerate(rows) if v == a], torch.int64))
                           for a in sorted(set(rows)) if a >= 0]
    elif case["op"] == "cache":
        T, H, D = case["T"], case["heads"], case["dim"]
        s["K"], s["V"] = _activations(g, T, H, D), _randn(g, T, H, D)
        slots, pages = _slots(case)
        s["slots"] = _int(slots)
        if own:
            svdq = _lib()
            s["cache"] = svdq.Kv4Cache(pages, case["page"], H, D, _prec(svdq, case))
    else:
        H, Hk, D, P = case["heads_q"], case["heads_kv"], case["dim"], case["page"]
        lens = _lengths(case)
        tables, pages = _tables(case)
        T = sum(q for q, _ in lens)
        s["q"] = _activations(g, T, H, D)
        s["table"] = _int(tables)
        starts = [0]
        for q, _ in lens:
            starts.append(starts[-1] + q)
        s["q_start"], s["kv_len"] = _int(starts), _int([kv for _, kv in lens])
        s["lens"], s["scale"] = lens, D ** -0.5
        if own:
            svdq = _lib()
            cache = svdq.Kv4Cache(pages, P, Hk, D, _prec(svdq, case))
        else:
            kq = torch.zeros(pages * P, Hk, D, dtype=torch.int8, device=DEV)
            vq = torch.zeros_like(kq)
            width = D // _group(case)
            ks = torch.zeros(pages * P, Hk, width, dtype=F32, device=DEV)
            vs = torch.zeros_like(ks)
        for b, (_, kv) in enumerate(lens):
            K, V = _activations(g, kv, Hk, D), _randn(g, kv, Hk, D)
            at = _slot_list(s["table"][b], kv, P)
            if own:
                svdq.kv4_append(cache, K, V, at.to(torch.int32))
            else:
                for x, q, sc in ((K, kq, ks), (V, vq, vs)):
                    q[at], sc[at] = _quantize(x, case)
        if own:
            s["cache"] = cache
            s["max_q"], s["max_kv"] = max(q for q, _ in lens), max(kv for _, kv in lens)
            s["work"] = svdq.kv4_attention_workspace(cache, T, len(lens), H, s["max_q"], s["max_kv"])
            s["out"] = torch.empty_like(s["q"])
        else:
            s["kq"], s["ks"], s["vq"], s["vs"] = kq, ks, vq, vs
    return s


def _prec(svdq, case):
    return svdq.INT4 if case["prec"] == "int4" else svdq.MXFP4


def _group(case):
    return 64 if case["prec"] == "int4" else 32


def _slot_list(table, kv, P):
    at = torch.arange(kv, device=DEV)
    return table[at // P].to(torch.int64) * P + at % P


# ------------------------------------------------------------- plain forms

def _plain_norm(v, kind, eps):
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    if kind != "none":
        v = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + eps)
    return v


def _run_norm(s):
    c, idx = s["case"], s["index"].long()
    t = _plain_norm(s["y"].float(), c["post"], 1e-6)
    if c["post"] != "none" and s["pw"] is not None:
        t = t * s["pw"].float()
    if s["gate"] is not None:
        t = t * s["gate"].float()[idx]
    r = s["r"].float() + c["alpha"] * t
    x = _plain_norm(r, c["pre"], 1e-6)
    if s["w"] is not None:
        x = x * s["w"].float()
    if s["b"] is not None:
        x = x + s["b"].float()
    if s["scale"] is not None:
        x = x * (1.0 + s["scale"].float()[idx]) + s["shift"].float()[idx]
    return r.to(s["r"].dtype), x.to(BF)


def _run_lora(s):
    Y = s["base"].float()
    for a, rows in s["groups"]:
        h = s["X"][rows].float() @ s["A"][a].float().t()
        Y[rows] += s["scale"][a] * (h @ s["B"][a].float().t())
    return Y.to(BF)


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _quantize(x, case):
    """Codes (INT4: integers; MXFP4: twice the E2M1 value) and fp32 scales of
    groups along the last dimension, the quotient formed in 64 bits."""
    g = _group(case)
    v = x.float().unflatten(-1, (-1, g))
    a = v.abs().amax(-1, keepdim=True)
    if case["prec"] == "int4":
        sc = (a.double() / 7.0).float()
        q = torch.round(v.double() / torch.where(sc == 0, torch.ones_like(sc), sc).double())
        return q.to(torch.int8).flatten(-2), sc.squeeze(-1)
    e = torch.frexp(a)[1] - 3                        # a = m 2^e', m in [1/2, 1): floor(log2 a) = e' - 1
    e = torch.where(a == 0, torch.full_like(e, -127), e).clamp(-127, 127)
    t = torch.ldexp(v.double(), -e)
    m = t.abs()
    i = ((m > 0.25).int() + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0)).long()
    grid = torch.tensor(_E2M1, device=x.device, dtype=F32)
    q = (2.0 * grid[i] * torch.sign(t)).to(torch.int8)
    return q.flatten(-2), torch.ldexp(torch.full_like(a, 0.5), e).squeeze(-1)


def _values(q, sc, case):
    return (q.unflatten(-1, (-1, _group(case))).float() * sc.unsqueeze(-1)).flatten(-2)


def _run_cache(s):
    return tuple(_values(*_quantize(x, s["case"]), s["case"]) for x in (s["K"], s["V"]))


def _mask(q, kv, causal, window):
    """Keys that query i of q sees, the queries being the last q of kv places."""
    i = torch.arange(q, device=DEV)[:, None] + (kv - q)
    j = torch.arange(kv, device=DEV)[None, :]
    keep = torch.ones(q, kv, dtype=torch.bool, device=DEV)
    if causal:
        keep &= j <= i
        if window > 0:
            keep &= j > i - window
    return keep


def _run_attend(s):
    c = s["case"]
    H, Hk, D, P = c["heads_q"], c["heads_kv"], c["dim"], c["page"]
    out = torch.empty(s["q"].shape, dtype=BF, device=DEV)
    at = 0
    for b, (q, kv) in enumerate(s["lens"]):
        slots = _slot_list(s["table"][b], kv, P)
        K = _values(s["kq"][slots], s["ks"][slots], c).permute(1, 2, 0).contiguous()       # Hk D kv
        V = _values(s["vq"][slots], s["vs"][slots], c).transpose(0, 1).contiguous()        # Hk kv D
        keep = _mask(q, kv, c["causal"], c["window"]) if c["causal"] else None
        Q = s["q"][at:at + q].float().view(q, Hk, H // Hk, D)
        for k in range(Hk):
            Qk = Q[:, k].transpose(0, 1).reshape(-1, D)
            S = ((Qk @ K[k]) * s["scale"]).view(H // Hk, q, kv)
            if keep is not None:
                S = S.masked_fill(~keep, -math.inf)
            E = torch.exp(S - S.amax(-1, keepdim=True))
            O = (E / E.sum(-1, keepdim=True)).view(-1, kv) @ V[k]
            out[at:at + q, k * (H // Hk):(k + 1) * (H // Hk)] = O.view(H // Hk, q, D).transpose(0, 1).to(BF)
        at += q
    return out


# ---------------------------------------------------------- library's calls

def _own_norm(s):
    svdq, c = _lib(), s["case"]
    kind = dict(none=svdq.NORM_NONE, rms=svdq.NORM_RMS, layer=svdq.NORM_LAYER)
    return svdq.residual_norm(s["r"], s["y"], gate=s["gate"], alpha=c["alpha"], post=kind[c["post"]],
                              post_w=s["pw"] if c["post"] != "none" else None, pre=kind[c["pre"]], pre_w=s["w"],
                              pre_b=s["b"], scale=s["scale"], shift=s["shift"],
                              mod_index=s["index"] if c["ragged"] else None, eps=1e-6)


def _own_lora(s):
    return _lib().lora_linear(s["X"], s["A"], s["B"], s["scale"], s["plan"], s["base"], Y=s["Y"], work=s["work"])


def _own_cache(s):
    svdq = _lib()
    svdq.kv4_append(s["cache"], s["K"], s["V"], s["slots"])
    return svdq.kv4_read(s["cache"], s["slots"])


def _own_attend(s):
    c = s["case"]
    return _lib().kv4_attention(s["q"], s["cache"], s["table"], s["q_start"], s["kv_len"], s["max_q"], s["max_kv"],
                                scale=s["scale"], causal=c["causal"], window=c["window"], out=s["out"],
                                work=s["work"])


def run(state):
    op = state["case"]["op"]
    if own:
        return dict(norm=_own_norm, lora=_own_lora, cache=_own_cache, attend=_own_attend)[op](state)
    return dict(norm=_run_norm, lora=_run_lora, cache=_run_cache, attend=_run_attend)[op](state)


# -------------------------------------------------------------------- work

def work(case):
    if case["op"] == "norm":
        M, D = case["M"], case["D"]
        vectors = case["images"] * (int(case["gate"]) + 2 * int(case["mod"])) + 2 * int(case["affine"])
        return dict(bytes=M * D * (2 * (4 if case["fp32"] else 2) + 4) + 2 * vectors * D, flops=12 * M * D)
    if case["op"] == "lora":
        rows = [a for a in _lora_rows(case) if a >= 0]
        K, N, R = case["K"], case["N"], case["R"]
        return dict(bytes=2 * len(rows) * K + 4 * case["M"] * N + 2 * len(set(rows)) * R * (K + N),
                    flops=2 * len(rows) * R * (K + N))
    sc = 4 / 64 if case["prec"] == "int4" else 1 / 32
    if case["op"] == "cache":
        n = 2 * case["T"] * case["heads"] * case["dim"]
        return dict(bytes=int(n * (2 + 4 + 2 * (0.5 + sc))), flops=8 * n)
    H, Hk, D = case["heads_q"], case["heads_kv"], case["dim"]
    rows = pairs = keys = 0
    for q, kv in _lengths(case):
        rows += q
        if case["causal"]:
            w = case["window"] if case["window"] > 0 else kv
            pairs += sum(min(kv - q + i + 1, w) for i in range(q))
            keys += min(kv, w + q - 1)
        else:
            pairs += q * kv
            keys += kv
    return dict(bytes=int(4 * rows * H * D + 2 * keys * Hk * D * (0.5 + sc)), flops=4 * D * H * pairs)


# ----------------------------------------------------- in 64 bits, apart

def exact(case, seed):
    return dict(norm=_exact_norm, lora=_exact_lora, cache=_exact_cache, attend=_exact_attend)[case["op"]](case, seed)


def _exact_inputs(case, seed):
    """The inputs alone (what `prepare` makes from the seed, without cache or plan)."""
    g = _gen(seed)
    if case["op"] == "cache":
        shape = (case["T"], case["heads"], case["dim"])
        return _activations(g, *shape), _randn(g, *shape)
    lens = _lengths(case)
    q = _activations(g, sum(n for n, _ in lens), case["heads_q"], case["dim"])
    kv = []
    for _, n in lens:
        shape = (n, case["heads_kv"], case["dim"])
        kv.append((_activations(g, *shape), _randn(g, *shape)))
    return q, kv


def _exact_norm(case, seed):
    s = prepare(case, seed)
    rows = torch.tensor(_norm_rows(case), device=DEV)
    r_out, x_out = [], []
    step = max(1, (1 << 24) // case["D"])

    def moments(z, kind):
        if kind == "none":
            return z
        mu = z.sum(1, keepdim=True) / z.shape[1] if kind == "layer" else torch.zeros_like(z[:, :1])
        var = ((z - mu) ** 2).sum(1, keepdim=True) / z.shape[1]
        return (z - mu) / torch.sqrt(var + 1e-6)

    for m in range(0, case["M"], step):
        at = rows[m:m + step]
        block = moments(s["y"][m:m + step].to(F64), case["post"])
        if case["post"] != "none" and case["affine"]:
            block = block * s["pw"].to(F64)
        weight = case["alpha"] * (s["gate"].to(F64)[at] if case["gate"] else 1.0)
        stream = s["r"][m:m + step].to(F64) + weight * block
        normed = moments(stream, case["pre"])
        if case["affine"]:
            normed = normed * s["w"].to(F64) + (s["b"].to(F64) if s["b"] is not None else 0.0)
        if case["mod"]:
            normed = normed + normed * s["scale"].to(F64)[at] + s["shift"].to(F64)[at]
        r_out.append(stream)
        x_out.append(normed)
    return torch.cat(r_out), torch.cat(x_out)


def _exact_lora(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    rows = torch.tensor(_lora_rows(case), device=DEV)
    out = s["base"].to(F64)
    for a in range(case["adapters"]):
        W = float(s["scale"][a]) * (s["B"][a].to(F64) @ s["A"][a].to(F64))     # the adapter as one matrix
        hit = torch.nonzero(rows == a).flatten()
        if hit.numel():
            out[hit] += s["X"][hit].to(F64) @ W.t()
    return out


def _exact_quantized(x, case):
    """The values that a cache holds for x, from the formats' definitions."""
    g = _group(case)
    v = x.to(F64).reshape(*x.shape[:-1], -1, g)
    top = v.abs().max(-1, keepdim=True).values
    if case["prec"] == "int4":
        step = (top / 7).to(F32).to(F64)
        q = torch.where(step > 0, v / step.clamp_min(1e-300), torch.zeros_like(v)).round()
        out = (q * step).to(F32).to(F64)
    else:
        power = torch.ldexp(torch.ones_like(top), torch.frexp(top.clamp_min(2.0 ** -125)).exponent - 3)
        # grid values next to v: 2 bits of significand, at least 1/2, at most 6; nearest, ties to the even index
        z = (v / power).abs().clamp_max(6.0)
        ulp = torch.where(z < 2, 0.5, torch.where(z < 4, 1.0, 2.0)).to(F64)
        out = torch.round(z / ulp) * ulp * torch.sign(v) * power
    return out.reshape(x.shape)


def _exact_cache(case, seed):
    return tuple(_exact_quantized(x, case) for x in _exact_inputs(case, seed))


def _exact_attend(case, seed):
    q_all, kv_all = _exact_inputs(case, seed)
    group = case["heads_q"] // case["heads_kv"]
    out = torch.zeros(q_all.shape, dtype=F64, device=DEV)
    at = 0
    for (q, kv), (K, V) in zip(_lengths(case), kv_all):
        K, V = _exact_quantized(K, case), _exact_quantized(V, case)
        place = torch.arange(kv - q, kv, device=DEV)
        key = torch.arange(kv, device=DEV)
        for h in range(case["heads_q"]):
            logits = q_all[at:at + q, h].to(F64) @ K[:, h // group].t().contiguous() / math.sqrt(case["dim"])
            if case["causal"]:
                hidden = key[None] > place[:, None]
                if case["window"]:
                    hidden |= key[None] <= place[:, None] - case["window"]
                logits[hidden] = -math.inf
            out[at:at + q, h] = torch.softmax(logits, -1) @ V[:, h // group].contiguous()
        at += q
    return out
