"""Operators of a decoder or image transformer whose linears, cache and steps
run in 4 bits: positions, drafted tokens, the gated MLP, linears of few rows.

Five families, each in a plain form (elementary torch operations in 32 bits,
64 where a rounding border or a far angle needs it) and as calls of the
library:

  rotate   rope_table + qk_norm_rope: cosines and sines of positions with
           several axes; norm and rotation of query and key heads
  append   kv4_rope_append: the same on the way into the 4-bit cache
  tree     kv4_tree_plan + kv4_tree_attention: attention of a tree of drafted
           tokens over the cache
  keep     kv4_keep_path: an accepted path of drafted tokens closes up
  linear   w4a4_linear_few (4-bit linear of few rows), w4a4_linear_gated (gate
           and up projection, activation and product)

`own` selects which one `run` computes.  Nothing outside a case and a seed
enters: the case fixes the sizes, lengths, positions and trees, the seed the
values.
"""
import math
import random

import torch

own = False

DEV = "cuda"
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
EPS = 1e-6


def _lib():
    import w4a4_rank_corrected_quantize_amd as svdq
    return svdq


# ------------------------------------------------------------------- cases

def _rotate(name, text, frames, high, wide, heads_q, heads_kv, dim, sections, layout="blocks", pairs="adjacent",
            theta=10000.0, norm=True, far=0):
    return dict(name=name, op="rotate", text=text, frames=frames, high=high, wide=wide, heads_q=heads_q,
                heads_kv=heads_kv, dim=dim, sections=sections, layout=layout, pairs=pairs, theta=theta, norm=norm,
                far=far)


def _append(name, prec, text, frames, high, wide, heads_q, heads_kv, dim, sections, page, layout="sections",
            pairs="halves", theta=1e6, norm=True, far=0, table=0, shape_seed=0):
    return dict(name=name, op="append", prec=prec, text=text, frames=frames, high=high, wide=wide, heads_q=heads_q,
                heads_kv=heads_kv, dim=dim, sections=sections, page=page, layout=layout, pairs=pairs, theta=theta,
                norm=norm, far=far, table=table, shape_seed=shape_seed)


def _tree(name, prec, B, heads_q, heads_kv, dim, page, nodes_min, nodes_max, kv_min, kv_max, chain=0.5, shape_seed=0):
    return dict(name=name, op="tree", prec=prec, B=B, heads_q=heads_q, heads_kv=heads_kv, dim=dim, page=page,
                nodes_min=nodes_min, nodes_max=nodes_max, kv_min=kv_min, kv_max=kv_max, chain=chain,
                shape_seed=shape_seed)


def _keep(name, prec, B, heads_kv, dim, page, nodes_min, nodes_max, kv_min, kv_max, chain=0.5, shape_seed=0):
    return dict(name=name, op="keep", prec=prec, B=B, heads_kv=heads_kv, dim=dim, page=page, nodes_min=nodes_min,
                nodes_max=nodes_max, kv_min=kv_min, kv_max=kv_max, chain=chain, shape_seed=shape_seed)


def _linear(name, prec, M, N, K, kind, bias=False):
    return dict(name=name, op="linear", prec=prec, M=M, N=N, K=K, kind=kind, bias=bias)


def listed():
    return [
        # a 1024 x 1024 image: 512 text tokens and 64 x 64 patches, three axes side by side in the head, neighbouring
        # channels paired
        _rotate("rotate_image", 512, 1, 64, 64, 24, 24, 128, "8,28,28"),
        # one token of a decoder: its row of a table of all positions, heads grouped
        _append("append_token", "mxfp4", 1, 0, 0, 0, 32, 8, 128, "64", 64, table=32768, far=20000),
        # a prompt with a short film between its text, sections of one frequency scale, halves paired
        _append("append_video", "int4", 301, 9, 22, 19, 28, 4, 128, "16,24,24", 32, shape_seed=3),
        # a short request checks eight drafted tokens
        _tree("tree_one", "int4", 1, 32, 8, 128, 16, 8, 8, 1000, 1000),
        # a batch of long requests checks up to 64 drafted tokens each
        _tree("tree_batch", "mxfp4", 16, 32, 8, 128, 64, 24, 64, 3000, 16384, shape_seed=7),
        # requests of all lengths, some without a prefix, chains beside wide trees, heads of 64
        _tree("tree_ragged", "int4", 9, 12, 4, 64, 32, 1, 130, 0, 5000, chain=0.8, shape_seed=11),
        # the accepted path of one request
        _keep("keep_one", "int4", 1, 8, 128, 16, 8, 8, 1000, 1000),
        # the accepted paths of a batch
        _keep("keep_batch", "mxfp4", 64, 8, 128, 64, 16, 64, 100, 1200, chain=0.9, shape_seed=5),
        # the MLP of one decoded token
        _linear("gated_token", "mxfp4", 1, 14336, 4096, "silu"),
        # the MLP over an image's tokens
        _linear("gated_image", "int4", 4608, 6912, 2560, "gelu_gated", bias=True),
        # the attention's projection of one decoded token
        _linear("few_token", "int4", 1, 6144, 4096, "none", bias=True),
        # the MLP's second projection over a request's drafted tokens
        _linear("few_draft", "mxfp4", 48, 4096, 11008, "none"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _sections(rng, pairs):
    """Pairs of one to three axes, multiples of 4."""
    n = rng.randint(1, 3)
    cuts = [0] + sorted(4 * v for v in rng.sample(range(1, pairs // 4), n - 1)) + [pairs]
    return ",".join(str(b - a) for a, b in zip(cuts, cuts[1:]))


def draw(rng):
    op = rng.choice(["rotate", "append", "tree", "tree", "keep", "few", "gated"])
    s = rng.randrange(1 << 30)
    prec = rng.choice(["int4", "mxfp4"])
    if op in ("rotate", "append"):
        dim = rng.choice([64, 128])
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.randint(1, 8)
        pairs = dim // 2 if rng.random() < 0.7 else dim // 4
        T = _log_int(rng, 1, 4608 * 48 * 128 // ((hq + 2 * hkv) * dim) // 2)
        wide = max(1, int(math.sqrt(T) * rng.uniform(0.3, 0.9)))
        high = max(1, int(T / wide * rng.uniform(0.2, 1.0)))
        frames = 1
        if high > 3 and rng.random() < 0.5:
            frames = rng.randint(2, high)
            high = max(1, high // frames)
        text = max(0, T - frames * high * wide)
        kw = dict(layout=rng.choice(["blocks", "sections", "interleaved"]), pairs=rng.choice(["adjacent", "halves"]),
                  theta=rng.choice([10000.0, 5e5, 1e6]), norm=rng.random() < 0.6, far=rng.choice([0, 0, 1000, 100000]))
        if op == "rotate":
            return _rotate("", text, frames, high, wide, hq, hkv, dim, _sections(rng, pairs), **kw)
        return _append("", prec, text, frames, high, wide, hq, hkv, dim, _sections(rng, pairs),
                       rng.choice([16, 32, 64, 128]), shape_seed=s, **kw)
    dim, hkv, page = rng.choice([64, 128]), rng.choice([1, 2, 4, 8]), rng.choice([16, 32, 64, 128])
    chain = rng.choice([0.0, 0.5, 0.9, 1.0])
    if op == "tree":
        nodes, B = _log_int(rng, 1, 128), _log_int(rng, 1, 16)
        hq = hkv * rng.choice([1, 2, 3, 4, 8])
        return _tree("", prec, B, hq, hkv, dim, page, rng.randint(1, nodes), nodes, 0,
                     _log_int(rng, 1, max(2, min(16000, (1 << 30) // (B * hq * nodes)))), chain, s)
    if op == "keep":
        nodes = _log_int(rng, 1, 128)
        return _keep("", prec, _log_int(rng, 1, 64), hkv, dim, page, rng.randint(1, nodes), nodes, 0, 1200, chain, s)
    step = 64 if prec == "int4" else 32
    K = step * _log_int(rng, 256 // step, 8192 // step)
    N = 8 * _log_int(rng, 32, 1792)
    if op == "few":
        return _linear("", prec, _log_int(rng, 1, 64), N, K, rng.choice(["none", "gelu"]), rng.random() < 0.5)
    N = min(N, 8 * (6912 * 2560 // (8 * K)) if K > 4096 else N)
    M = _log_int(rng, 1, max(1, min(4608, 4608 * 6912 * 2560 // (N * K))))
    return _linear("", prec, M, N, K, rng.choice(["silu", "gelu_gated"]), rng.random() < 0.5)


# --------------------------------------------- sizes that a case stands for

def _positions(case):
    """Positions of the tokens on every axis: text counts on all axes alike, a picture's or film's patches have their
    frame, row and column from there."""
    axes = len(case["sections"].split(","))
    n, before = case["text"], case["text"] // 2
    out = [(case["far"] + i,) * 3 for i in range(before)]
    at = case["far"] + before
    for t in range(case["frames"]):
        out += [(at + t, at + y, at + x) for y in range(case["high"]) for x in range(case["wide"])]
    at += max(case["frames"], case["high"], case["wide"])
    out += [(at + i,) * 3 for i in range(n - before)]
    return [p[:axes] for p in out]


def _tokens(case):
    return case["text"] + case["frames"] * case["high"] * case["wide"]


def _axis_and_frequency(case):
    """Axis and frequency of every pair of channels.  blocks: an axis has a run of pairs with frequencies of its own,
    theta^(-j / n); sections: runs of pairs, the frequencies falling over all of them; interleaved: the axes in turn
    while their pairs last, the rest the first axis."""
    parts = [int(v) for v in case["sections"].split(",")]
    total, theta = sum(parts), case["theta"]
    if case["layout"] == "blocks":
        return ([a for a, n in enumerate(parts) for _ in range(n)],
                [theta ** (-j / n) for n in parts for j in range(n)])
    if case["layout"] == "sections":
        axis = [a for a, n in enumerate(parts) for _ in range(n)]
    else:
        axis = [p % len(parts) if p // len(parts) < parts[p % len(parts)] else 0 for p in range(total)]
    return axis, [theta ** (-p / total) for p in range(total)]


def _slots(case):
    """Slots of the tokens: pages in a shuffled order; and the number of pages."""
    rng = random.Random(case["shape_seed"])
    P, T = case["page"], _tokens(case)
    pages = -(-T // P) + 3
    order = list(range(pages))
    rng.shuffle(order)
    return [order[t // P] * P + t % P for t in range(T)], pages


def _trees(case):
    """(parents, prefix) of every sequence: a node's parent comes before it, -1 is the last token of the prefix."""
    rng = random.Random(case["shape_seed"])
    out = []
    for _ in range(case["B"]):
        n = rng.randint(case["nodes_min"], case["nodes_max"])
        parent = [i - 1 if rng.random() < case["chain"] else rng.randint(-1, i - 1) for i in range(n)]
        out.append((parent, rng.randint(case["kv_min"], case["kv_max"])))
    return out


def _paths(case):
    """The accepted nodes of every sequence: from the root to some node."""
    rng = random.Random(case["shape_seed"] + 2)
    out = []
    for parent, _ in _trees(case):
        node, path = rng.randrange(len(parent)), []
        while node >= 0:
            path.append(node)
            node = parent[node]
        out.append(path[::-1])
    return out


def _tables(case):
    rng = random.Random(case["shape_seed"] + 1)
    P = case["page"]
    need = [-(-(prefix + len(parent)) // P) for parent, prefix in _trees(case)]
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


def _group(case):
    return 64 if case["prec"] == "int4" else 32


def _prec(svdq, case):
    return svdq.INT4 if case["prec"] == "int4" else svdq.MXFP4


def _codes(g, case, rows, K, size):
    """Packed codes and scales of a [rows][K] matrix as the packing and activation steps leave them (the largest of a
    group near the largest code), its values about normal with deviation `size`."""
    x = torch.randn(rows, K, generator=g, device=DEV, dtype=F32)
    G = K // _group(case)
    spread = torch.rand(rows, G, generator=g, device=DEV)
    if case["prec"] == "int4":
        mag = (x.abs() * 2.8).round_().clamp_(max=7)
        scale = size / 2.8 * (0.75 + 0.5 * spread)
    else:
        grid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
        mag = torch.bucketize(x.abs() * 2.0, grid)
        scale = (127 + math.floor(math.log2(size / 2.0)) + 2.0 * spread).to(torch.uint8)
    code = mag.to(torch.uint8) + 8 * (x < 0).to(torch.uint8)
    return code[:, 0::2] + 16 * code[:, 1::2], scale


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case=case)
    if op in ("rotate", "append"):
        T, D = _tokens(case), case["dim"]
        Hq, Hk = case["heads_q"], case["heads_kv"]
        qkv = _activations(g, T, (Hq + 2 * Hk) * D)          # one projection's output
        s["Q"], s["K"], s["V"] = (t.unflatten(1, (-1, D)) for t in qkv.split((Hq * D, Hk * D, Hk * D), 1))
        s["wq"] = (1.0 + 0.2 * torch.randn(D, generator=g, device=DEV)).to(BF) if case["norm"] else None
        s["wk"] = (1.0 + 0.2 * torch.randn(D, generator=g, device=DEV)).to(BF) if case["norm"] else None
        axis, freq = _axis_and_frequency(case)
        s["axis"], s["freq"] = _int(axis), torch.tensor(freq, dtype=F64, device=DEV)
        s["pos"] = _int(_positions(case))
    if op == "append":
        # the step's table, made once for all layers; or that of all positions, made once
        if case["table"]:
            s["index"] = s["pos"][:, 0].contiguous()
            angle = torch.arange(case["table"], device=DEV).to(F64)[:, None] * s["freq"]
        else:
            s["index"] = None
            angle = s["pos"][:, s["axis"].long()].to(F64) * s["freq"]
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        slots, pages = _slots(case)
        s["slots"] = _int(slots)
        if own:
            svdq = _lib()
            s["cache"] = svdq.Kv4Cache(pages, case["page"], Hk, D, _prec(svdq, case))
    elif op in ("tree", "keep"):
        trees, P = _trees(case), case["page"]
        tables, pages = _tables(case)
        counts = [len(parent) for parent, _ in trees]
        starts = [0]
        for n in counts:
            starts.append(starts[-1] + n)
        T = starts[-1]
        s["counts"], s["prefix"] = counts, [prefix for _, prefix in trees]
        s["table"], s["q_start"] = _int(tables), _int(starts)
        s["parent"] = _int([p for parent, _ in trees for p in parent])
        s["kv_len"] = _int([prefix + len(parent) for parent, prefix in trees])
        Hk, D = case["heads_kv"], case["dim"]
        s["max_q"], s["max_kv"] = max(counts), max(p + n for p, n in zip(s["prefix"], counts))
        if own:
            svdq = _lib()
            s["cache"] = svdq.Kv4Cache(pages, P, Hk, D, _prec(svdq, case))
        if op == "tree":
            s["Q"] = _activations(g, T, case["heads_q"], D)
            keys = [prefix + n for prefix, n in zip(s["prefix"], counts)]
            at = _int([tables[b][i // P] * P + i % P for b, n in enumerate(keys) for i in range(n)])
            K, V = _activations(g, len(at), Hk, D), _randn(g, len(at), Hk, D)
            if own:
                svdq.kv4_append(s["cache"], K, V, at)
                s["work"] = svdq.kv4_attention_workspace(s["cache"], T, len(counts), case["heads_q"], s["max_q"],
                                                         s["max_kv"])
                s["out"], s["lse"] = torch.empty_like(s["Q"]), torch.empty(T, case["heads_q"], device=DEV)
            else:
                for name, x in (("k", K), ("v", V)):
                    q, sc = _quantize(x, case)
                    s[name + "q"] = torch.zeros(pages * P, Hk, D, dtype=torch.int8, device=DEV)
                    s[name + "s"] = torch.zeros(pages * P, Hk, D // _group(case), device=DEV)
                    s[name + "q"][at.long()], s[name + "s"][at.long()] = q, sc
        else:
            s["K"], s["V"] = _activations(g, T, Hk, D), _randn(g, T, Hk, D)
            paths = _paths(case)
            longest = max(len(p) for p in paths)
            s["path"] = _int([p + [-1] * (longest - len(p)) for p in paths])
            place = [(b, s["prefix"][b] + i) for b, n in enumerate(counts) for i in range(n)]
            s["slots"] = _int([tables[b][i // P] * P + i % P for b, i in place])
            kept = [(b, s["prefix"][b] + i) for b, p in enumerate(paths) for i in range(len(p))]
            s["kept"] = _int([tables[b][i // P] * P + i % P for b, i in kept])
    elif op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        rows = 2 * N if _gated(case) else N
        s["xq"], s["xscale"] = _codes(g, case, M, K, 1.0)
        s["wq"], s["wscale"] = _codes(g, case, rows, K, K ** -0.5)
        s["h"] = torch.randn(M, 32, generator=g, device=DEV)
        s["up"] = _randn(g, rows, 32, scale=0.5 * 32 ** -0.5)
        s["bias"] = _randn(g, rows, scale=0.2) if case["bias"] else None
        s["Y"] = torch.empty(M, N, dtype=BF, device=DEV)
    return s


def _gated(case):
    return case["kind"] in ("silu", "gelu_gated")


# ------------------------------------------------------------- plain forms

_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _quantize(x, case):
    """Codes (INT4: integers; MXFP4: twice the E2M1 value) and fp32 scales of groups along the last dimension, the
    quotient formed in 64 bits."""
    v = x.float().unflatten(-1, (-1, _group(case)))
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
    q = (2.0 * torch.tensor(_E2M1, device=x.device)[i] * torch.sign(t)).to(torch.int8)
    return q.flatten(-2), torch.ldexp(torch.full_like(a, 0.5), e).squeeze(-1)


def _values(q, sc, case):
    return (q.unflatten(-1, (-1, _group(case))).float() * sc.unsqueeze(-1)).flatten(-2)


def _rotated(x, w, cos, sin, case):
    """Norm over the head and rotation in 64 bits (what follows may round it to 4 bits); cos and sin [T][pairs]."""
    u = x.double()
    if w is not None:
        u = u * torch.rsqrt((u * u).mean(-1, keepdim=True) + EPS) * w.double()
    n = cos.shape[1]
    c, s = cos.double()[:, None], sin.double()[:, None]
    if case["pairs"] == "adjacent":
        a, b = u[..., 0:2 * n:2], u[..., 1:2 * n:2]
        r = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = u[..., :n], u[..., n:2 * n]
        r = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((r, u[..., 2 * n:]), -1).float().to(BF)


def _run_rotate(s):
    angle = s["pos"][:, s["axis"].long()].double() * s["freq"]
    cos, sin = angle.cos().float(), angle.sin().float()
    return (cos, sin, _rotated(s["Q"], s["wq"], cos, sin, s["case"]),
            _rotated(s["K"], s["wk"], cos, sin, s["case"]))


def _run_append(s):
    c = s["case"]
    cos, sin = s["cos"], s["sin"]
    if s["index"] is not None:
        cos, sin = cos[s["index"].long()], sin[s["index"].long()]
    K = _rotated(s["K"], s["wk"], cos, sin, c)
    return (_rotated(s["Q"], s["wq"], cos, sin, c),) + tuple(_values(*_quantize(x, c), c) for x in (K, s["V"]))


def _ancestors(parent, valid):
    """[B][n][n]: node j lies on the way from the root to node i, i itself included; parents [B][n]."""
    n = parent.shape[1]
    node = torch.arange(n, device=DEV)
    step = (parent[:, :, None] == node) & valid[:, :, None]
    self = (node[:, None] == node) & valid[:, :, None]
    return torch.matrix_power((step | self).double(), n) > 0       # binomials: every entry below 2^n


def _run_tree(s):
    c = s["case"]
    H, Hk, D, P = c["heads_q"], c["heads_kv"], c["dim"], c["page"]
    B, n, kv = len(s["counts"]), s["max_q"], s["max_kv"]
    count, prefix = s["q_start"][1:] - s["q_start"][:-1], s["kv_len"] - (s["q_start"][1:] - s["q_start"][:-1])
    node, key = torch.arange(n, device=DEV), torch.arange(kv, device=DEV)
    valid = node < count[:, None]
    row = (s["q_start"][:-1, None] + node).clamp(max=len(s["parent"]) - 1).long()
    above = _ancestors(s["parent"][row], valid)
    # the drafted tokens' places, and the mask in words of 32
    position = prefix[:, None] + above.sum(-1) - 1
    place = (prefix[:, None] + node).clamp(max=kv - 1)
    slots = s["table"].gather(1, (place // P).long()) * P + place % P
    words = torch.nn.functional.pad(above, (0, -n % 32)).unflatten(-1, (-1, 32)).long()
    mask = (words << torch.arange(32, device=DEV)).sum(-1)
    mask = torch.where(mask >= 1 << 31, mask - (1 << 32), mask).int()
    # attention over the padded batch
    at = (s["table"][:, key // P].long() * P + key % P).clamp(min=0)
    K = _values(s["kq"][at], s["ks"][at], c).permute(0, 2, 3, 1).contiguous()            # B Hk D kv
    V = _values(s["vq"][at], s["vs"][at], c).transpose(1, 2).contiguous()                # B Hk kv D
    Q = s["Q"][row].float().view(B, n, Hk, H // Hk, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, -1, D)
    S = ((Q @ K) * D ** -0.5).view(B, Hk, H // Hk, n, kv)
    drafted = (key - prefix[:, None]).long()
    seen = above.gather(2, drafted.clamp(0, n - 1)[:, None].expand(B, n, kv)) & (drafted < count[:, None])[:, None]
    seen |= (drafted < 0)[:, None]
    S = S.masked_fill(~seen[:, None, None], -math.inf)
    top = S.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    E = torch.exp(S - top)
    total = E.sum(-1, keepdim=True)
    O = ((E / total).view(B, Hk, -1, kv) @ V).view(B, Hk, H // Hk, n, D).permute(0, 3, 1, 2, 4).reshape(B, n, H, D)
    lse = (top + torch.log(total)).squeeze(-1).permute(0, 3, 1, 2).reshape(B, n, H)
    return position[valid].int(), slots[valid].int(), mask[valid], O[valid].to(BF), lse[valid]


def _run_keep(s):
    c = s["case"]
    ok = s["path"] >= 0
    row = (s["q_start"][:-1, None] + s["path"])[ok].long()
    length = s["kv_len"] - (s["q_start"][1:] - s["q_start"][:-1]) + ok.sum(1)
    return (length.int(),) + tuple(_values(*_quantize(x[row], c), c) for x in (s["K"], s["V"]))


def _decode(q, sc, case):
    """fp32 values of packed codes."""
    code = torch.stack((q & 15, q >> 4), -1).flatten(-2)
    grid = range(8) if case["prec"] == "int4" else _E2M1
    value = torch.tensor([float(v) for v in grid] + [-float(v) for v in grid], device=DEV)[code.int()]
    if case["prec"] == "mxfp4":
        sc = torch.ldexp(torch.ones_like(sc, dtype=F32), sc.int() - 127)
    return (value.unflatten(-1, (-1, _group(case))) * sc.unsqueeze(-1)).flatten(-2)


def _gelu_tanh(y):
    return 0.5 * y * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (y + 0.044715 * y * y * y)))


def _run_linear(s):
    c = s["case"]
    y = _decode(s["xq"], s["xscale"], c) @ _decode(s["wq"], s["wscale"], c).t() + s["h"] @ s["up"].float().t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    if _gated(c):
        gate, up = y[:, :c["N"]], y[:, c["N"]:]
        y = (gate / (1.0 + torch.exp(-gate)) if c["kind"] == "silu" else _gelu_tanh(gate)) * up
    elif c["kind"] == "gelu":
        y = _gelu_tanh(y)
    return y.to(BF)


# ---------------------------------------------------------- library's calls

def _own_rotate(s):
    svdq, c = _lib(), s["case"]
    cos, sin = svdq.rope_table(s["pos"], s["freq"], s["axis"])
    style = svdq.ROPE_ADJACENT if c["pairs"] == "adjacent" else svdq.ROPE_HALVES
    Q, K = svdq.qk_norm_rope(s["Q"], s["K"], cos, sin, style=style, norm_q=s["wq"], norm_k=s["wk"], eps=EPS)
    return cos, sin, Q, K


def _own_append(s):
    svdq, c = _lib(), s["case"]
    style = svdq.ROPE_ADJACENT if c["pairs"] == "adjacent" else svdq.ROPE_HALVES
    Q = svdq.kv4_rope_append(s["cache"], s["Q"], s["K"], s["V"], s["cos"], s["sin"], s["slots"], style=style,
                             index=s["index"], norm_q=s["wq"], norm_k=s["wk"], eps=EPS)
    return (Q,) + tuple(svdq.kv4_read(s["cache"], s["slots"]))


def _own_tree(s):
    svdq = _lib()
    mask, position, slots = svdq.kv4_tree_plan(s["cache"], s["parent"], s["q_start"], s["kv_len"], s["table"],
                                               s["max_q"])
    out = svdq.kv4_tree_attention(s["Q"], s["cache"], s["table"], s["q_start"], s["kv_len"], mask, s["max_q"],
                                  s["max_kv"], out=s["out"], lse=s["lse"], work=s["work"])
    return position, slots, mask, out, s["lse"]


def _own_keep(s):
    svdq = _lib()
    svdq.kv4_append(s["cache"], s["K"], s["V"], s["slots"])
    length = svdq.kv4_keep_path(s["cache"], s["path"], s["q_start"], s["kv_len"], s["table"])
    return (length,) + tuple(svdq.kv4_read(s["cache"], s["kept"]))


def _own_linear(s):
    svdq, c = _lib(), s["case"]
    args = (s["xq"], s["xscale"], s["h"], s["wq"], s["wscale"], s["up"], s["bias"], _prec(svdq, c))
    if _gated(c):
        act = svdq.ACT_SILU if c["kind"] == "silu" else svdq.ACT_GELU_TANH
        return svdq.w4a4_linear_gated(*args, act=act, Y=s["Y"])
    epi = svdq.EPI_GELU_TANH if c["kind"] == "gelu" else svdq.EPI_NONE
    return svdq.w4a4_linear_few(*args, epi=epi, Y=s["Y"])


def run(state):
    op = state["case"]["op"]
    if own:
        return dict(rotate=_own_rotate, append=_own_append, tree=_own_tree, keep=_own_keep,
                    linear=_own_linear)[op](state)
    return dict(rotate=_run_rotate, append=_run_append, tree=_run_tree, keep=_run_keep, linear=_run_linear)[op](state)


# -------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        rows = 2 * N if _gated(case) else N
        per = 0.5 + (4 / 64 if case["prec"] == "int4" else 1 / 32)
        return dict(bytes=int((M + rows) * K * per + 128 * M + (66 if case["bias"] else 64) * rows + 2 * M * N),
                    flops=2 * M * rows * (K + 32))
    Hk, D = case["heads_kv"], case["dim"]
    if op in ("rotate", "append"):
        T, Hq = _tokens(case), case["heads_q"]
        pairs = sum(int(v) for v in case["sections"].split(","))
        axes = len(case["sections"].split(","))
        if op == "rotate":
            return dict(bytes=T * (4 * (Hq + Hk) * D + 8 * pairs + 4 * axes) + 12 * pairs,
                        flops=T * (8 * (Hq + Hk) * D + 4 * pairs))
        held = 0.5 + (4 / 64 if case["prec"] == "int4" else 1 / 32)
        return dict(bytes=int(T * (4 * Hq * D + 2 * Hk * D * (2 + 2 * held + 4) + 8 * pairs + 4)),
                    flops=T * (8 * (Hq + Hk) * D + 16 * Hk * D))
    held = 0.5 + (4 / 64 if case["prec"] == "int4" else 1 / 32)
    trees = _trees(case)
    T = sum(len(parent) for parent, _ in trees)
    if op == "keep":
        kept = sum(len(p) for p in _paths(case))
        return dict(bytes=int(2 * T * Hk * D * (2 + held) + 2 * kept * Hk * D * (3 * held + 4)),
                    flops=16 * T * Hk * D)
    H = case["heads_q"]
    keys = sum(len(parent) + prefix for parent, prefix in trees)
    pairs = 0
    for parent, prefix in trees:
        depth = []
        for p in parent:
            depth.append(1 if p < 0 else depth[p] + 1)
        pairs += len(parent) * prefix + sum(depth)
    return dict(bytes=int(4 * T * H * D + 4 * T * H + 2 * keys * Hk * D * held + 16 * T), flops=4 * D * H * pairs)


# ----------------------------------------------------- in 64 bits, apart

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return dict(rotate=_exact_rotate, append=_exact_append, tree=_exact_tree, keep=_exact_keep,
                linear=_exact_linear)[case["op"]](case, s)


def _exact_turn(x, weight, angle_cos, angle_sin, case):
    """x as complex numbers, one per pair, times e^(i angle)."""
    z = x.to(F64)
    if weight is not None:
        z = z / torch.sqrt((z ** 2).sum(-1, keepdim=True) / z.shape[-1] + EPS) * weight.to(F64)
    n = angle_cos.shape[1]
    turned = z[..., :2 * n]
    turned = turned.unflatten(-1, (n, 2)) if case["pairs"] == "adjacent" else turned.unflatten(-1, (2, n)).transpose(-1, -2)
    turned = torch.view_as_complex(turned.contiguous()) * torch.complex(angle_cos, angle_sin)[:, None]
    turned = torch.view_as_real(turned)
    turned = turned if case["pairs"] == "adjacent" else turned.transpose(-1, -2)
    return torch.cat((turned.flatten(-2), z[..., 2 * n:]), -1)


def _exact_angles(case):
    axis, freq = _axis_and_frequency(case)
    pos = torch.tensor(_positions(case), dtype=F64, device=DEV)
    return pos[:, axis] * torch.tensor(freq, dtype=F64, device=DEV)


def _exact_rotate(case, s):
    angle = _exact_angles(case)
    return (torch.cos(angle), torch.sin(angle), _exact_turn(s["Q"], s["wq"], torch.cos(angle), torch.sin(angle), case),
            _exact_turn(s["K"], s["wk"], torch.cos(angle), torch.sin(angle), case))


def _exact_held(x, case):
    """The values that a cache holds for bf16 x, from the formats' definitions."""
    v = x.to(F64).reshape(*x.shape[:-1], -1, _group(case))
    top = v.abs().max(-1, keepdim=True).values
    if case["prec"] == "int4":
        step = (top / 7).to(F32).to(F64)
        out = (torch.where(step > 0, v / step.clamp_min(1e-300), torch.zeros_like(v)).round() * step).to(F32).to(F64)
    else:
        power = torch.ldexp(torch.ones_like(top), torch.frexp(top.clamp_min(2.0 ** -125)).exponent - 3)
        z = (v / power).abs().clamp_max(6.0)
        ulp = torch.where(z < 2, 0.5, torch.where(z < 4, 1.0, 2.0)).to(F64)
        out = torch.round(z / ulp) * ulp * torch.sign(v) * power
    return out.reshape(x.shape)


def _exact_append(case, s):
    # the tables are inputs, in 32 bits
    at = s["index"].long() if s["index"] is not None else torch.arange(s["cos"].shape[0], device=DEV)
    c, n = s["cos"][at].to(F64), s["sin"][at].to(F64)
    K = _exact_turn(s["K"], s["wk"], c, n, case).to(F32).to(BF)
    return _exact_turn(s["Q"], s["wq"], c, n, case), _exact_held(K, case), _exact_held(s["V"], case)


def _exact_tree(case, s):
    """Sequence by sequence, the ancestors by walking up."""
    H, G, P = case["heads_q"], case["heads_q"] // case["heads_kv"], case["page"]
    out, lse, at = [], [], 0
    for b, (parent, prefix) in enumerate(_trees(case)):
        n, kv = len(parent), len(parent) + prefix
        hidden = torch.ones(n, kv, dtype=torch.bool)
        hidden[:, :prefix] = False
        for i in range(n):
            j = i
            while j >= 0:
                hidden[i, prefix + j] = False
                j = parent[j]
        hidden = hidden.to(DEV)
        place = torch.arange(kv, device=DEV)
        slot = s["table"][b, place // P].long() * P + place % P
        held = [(q[slot].to(F64).unflatten(-1, (-1, _group(case))) * sc[slot].to(F64)[..., None]).flatten(-2)
                for q, sc in ((s["kq"], s["ks"]), (s["vq"], s["vs"]))]
        K, V = (x.transpose(0, 1).repeat_interleave(G, 0) for x in held)                 # H kv D
        for_q = s["Q"][at:at + n].to(F64).transpose(0, 1)                                # H n D
        o, l = torch.empty_like(for_q), torch.empty(H, n, dtype=F64, device=DEV)
        for h in range(H):
            logits = (for_q[h] @ K[h].t().contiguous() / math.sqrt(case["dim"])).masked_fill(hidden, -math.inf)
            o[h], l[h] = torch.softmax(logits, -1) @ V[h], torch.logsumexp(logits, -1)
        out.append(o.transpose(0, 1))
        lse.append(l.t())
        at += n
    return None, None, None, torch.cat(out), torch.cat(lse)


def _exact_keep(case, s):
    rows, start = [], 0
    for (parent, _), path in zip(_trees(case), _paths(case)):
        rows += [start + p for p in path]
        start += len(parent)
    return None, _exact_held(s["K"][rows], case), _exact_held(s["V"][rows], case)


def _exact_linear(case, s):
    table = [0, 1, 2, 3, 4, 5, 6, 7] if case["prec"] == "int4" else [0, 0.5, 1, 1.5, 2, 3, 4, 6]

    def matrix(q, sc):
        out = torch.empty(q.shape[0], case["K"], dtype=F64, device=DEV)
        for half, code in ((0, q & 15), (1, q >> 4)):
            mag = torch.tensor(table, dtype=F64, device=DEV)[(code & 7).long()]
            out[:, half::2] = torch.where(code >= 8, -mag, mag)
        size = sc.to(F64) if case["prec"] == "int4" else 2.0 ** (sc.to(F64) - 127)
        return out * size.repeat_interleave(_group(case), 1)

    X, rows = matrix(s["xq"], s["xscale"]), []
    for n in range(0, s["wq"].shape[0], 4096):
        part = X @ matrix(s["wq"][n:n + 4096], s["wscale"][n:n + 4096]).t()
        rows.append(part + s["h"].to(F64) @ s["up"][n:n + 4096].to(F64).t())
    y = torch.cat(rows, 1)
    if case["bias"]:
        y = y + s["bias"].to(F64)
    if case["kind"] == "none":
        return y
    z = y[:, :case["N"]]
    act = z * torch.sigmoid(z) if case["kind"] == "silu" else torch.nn.functional.gelu(z, approximate="tanh")
    return act * y[:, case["N"]:] if _gated(case) else act
