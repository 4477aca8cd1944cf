"""Cases that measure the operators around the decode step: the per-head norms and rotation that make its rows
(``csa_qk_norm_rope``), the cache held in 4 bits (``csa_kv4_append``, ``csa_kv4_unpack``) and the attention that reads it
(``csa_kv4_decode``).

With ``own`` false, ``run`` computes an operator from elementary torch operations; with ``own`` true it makes the calls a
user makes of the library.  Lengths live on the device, as in a decode loop replayed from a CUDA graph.

The 4-bit cache of one (sequence, KV head), in blocks of 64 tokens:
  K4      [64][d/2] per block, even channel in the low nibble; per channel the block's minimum m and step D = (max - min) / 15
  bounds  [2][d] per block: m, D
  V4      [d][32] per block: row = channel, nibble of token t = 32 i + 16 u + 8 v + 2 w + e at place 16 w + 8 i + 4 e + 2 u + v
  vscale  [64][2] per block: each token's minimum and step over its channels
  Kt, Vt  [64][d]: the rows of the incomplete last block, unquantised
"""
import math

import numpy as np
import torch

own = False

BLOCK = 64
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step's new tokens of a batch, written into the 16-bit cache the decode entry points read
        dict(name="rope tokens", op="rope", B=32, T=1, Hq=32, Hkv=8, d=128, dtype="bf16", rot=128, interleaved=False, cache=True,
             n_max=1024, ragged=True),
        # a prompt of 16K tokens in two sequences
        dict(name="rope prompt", op="rope", B=2, T=8192, Hq=32, Hkv=8, d=128, dtype="bf16", rot=128, interleaved=False, cache=True,
             n_max=8448, ragged=False),
        # half of the channels rotated in adjacent pairs, f32, an odd ragged chunk far into the context, rows kept apart from the cache
        dict(name="rope f32 chunk", op="rope", B=3, T=333, Hq=16, Hkv=8, d=64, dtype="f32", rot=32, interleaved=True, cache=False,
             n_max=1000000, ragged=True),
        # one decode step's new tokens into the 4-bit cache, and the block that holds each read back
        dict(name="append tokens", op="append", B=64, T=1, Hkv=8, d=128, dtype="bf16", n_max=2048, ragged=True),
        # prompt chunks of up to 8K tokens appended at odd places and read back for attention within the chunk
        dict(name="append prompt", op="append", B=4, T=8191, Hkv=8, d=128, dtype="bf16", n_max=12288, ragged=True),
        # a cached prefix of 32K tokens read back as 16-bit rows
        dict(name="unpack prefix", op="unpack", B=4, rows=32768, Hkv=8, d=128, dtype="bf16", n_max=32800, ragged=False),
        # the last rows of each sequence of a batch, full precision ones among them
        dict(name="unpack last rows", op="unpack", B=16, rows=100, Hkv=8, d=64, dtype="f32", n_max=1200, ragged=True),
        # one short conversation: latency counts
        dict(name="decode short", op="decode", B=1, T=1, Hq=32, Hkv=8, d=128, dtype="bf16", n_max=1000, ragged=False),
        # a serving batch of uneven lengths, eight query heads to a KV head
        dict(name="decode batch", op="decode", B=64, T=1, Hq=64, Hkv=8, d=128, dtype="bf16", n_max=8191, ragged=True),
        # several drafted tokens of each sequence checked at once
        dict(name="decode drafts", op="decode", B=8, T=6, Hq=32, Hkv=8, d=128, dtype="bf16", n_max=20000, ragged=True),
        # f32 queries, small heads
        dict(name="decode f32", op="decode", B=2, T=1, Hq=16, Hkv=8, d=64, dtype="f32", n_max=30001, ragged=True),
        # the benchmark's step: 128K tokens, four sequences, 32/8 heads
        dict(name="decode long", op="decode", B=4, T=1, Hq=32, Hkv=8, d=128, dtype="bf16", n_max=131072, ragged=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "unpack", "decode", "decode"])
    d, dtype = rng.choice([64, 128]), rng.choice(["bf16", "bf16", "f32"])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    Hq = Hkv * rng.choice([1, 2, 4, 8])
    B = _log(rng, 1, 64)
    ragged = rng.random() < 0.75
    if op == "rope":
        T = _log(rng, 1, max(1, min(8192, (1 << 17) // (B * max(1, Hq // 4)))))
        return dict(op=op, B=B, T=T, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, rot=rng.choice([d, d, d // 2, d // 4, 24]),
                    interleaved=rng.random() < 0.4, cache=rng.random() < 0.5,
                    n_max=T + _log(rng, 1, max(1, min(4096, (1 << 18) // (B * Hkv)))), ragged=ragged)
    if op == "append":
        T = _log(rng, 1, max(1, min(8191, (1 << 17) // (B * Hkv))))
        return dict(op=op, B=B, T=T, Hkv=Hkv, d=d, dtype=dtype, n_max=T + 128 + _log(rng, 1, 2048), ragged=ragged)
    if op == "unpack":
        rows = _log(rng, 1, max(1, min(32768, (1 << 19) // (B * Hkv))))
        return dict(op=op, B=B, rows=rows, Hkv=Hkv, d=d, dtype=dtype, n_max=rows + _log(rng, 1, 512), ragged=ragged)
    T = rng.choice([1, 1, 1, 2, 3, 5, 8, 16])
    T = min(T, 64 // (Hq // Hkv))
    n = _log(rng, 1, max(1, min(131072, (1 << 21) // (B * Hkv))))
    return dict(op=op, B=B, T=T, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, n_max=n, ragged=ragged)


def _lens(case, seed):
    """Lengths of the sequences after this pass's new tokens, and how many of those there are, on the host."""
    r = np.random.RandomState(seed % (1 << 31))
    B, n = case["B"], case["n_max"]
    op = case["op"]
    if op in ("rope", "append"):
        T = case["T"]
        new = r.randint(T // 2 + 1, T + 1, B) if case["ragged"] else np.full(B, T)
        new[0] = T
        # room for the block-aligned rows around the new ones
        top = n if op == "rope" else n - 2 * BLOCK
        return new + r.randint(0, max(1, top - T + 1), B), new
    if op == "unpack":
        rows = case["rows"]
        new = r.randint(rows // 2 + 1, rows + 1, B) if case["ragged"] else np.full(B, rows)
        return new + r.randint(0, n - rows + 1, B), new
    lens = r.randint(n // 8 + 1, n + 1, B) if case["ragged"] else np.full(B, n)
    lens[0] = n
    new = np.minimum(lens, r.randint(1, case["T"] + 1, B) if case["ragged"] else case["T"])
    return lens, new


def work(case):
    B, d, esz = case["B"], case["d"], 2 if case["dtype"] == "bf16" else 4
    lens, new = _lens(case, 7)
    code = d + 8 * d / BLOCK + 8  # bytes of one quantised token of one KV head: K and V codes, bounds, scales
    op = case["op"]
    if op == "rope":
        row = case["Hq"] + 2 * case["Hkv"]
        return {"bytes": 2.0 * esz * d * row * float(new.sum()), "flops": 10.0 * d * (case["Hq"] + case["Hkv"]) * float(new.sum())}
    rows = float(new.sum()) * case["Hkv"]
    if op == "append":  # rows in, codes out (full precision while their block is incomplete), rows read back
        if case["T"] == 1:
            return {"bytes": rows * 6 * d * esz, "flops": 0}
        return {"bytes": rows * (4 * d * esz + 2 * code), "flops": 12.0 * d * rows}
    if op == "unpack":
        return {"bytes": rows * (2 * d * esz + code), "flops": 4.0 * d * rows}
    q = float(new.sum()) * case["Hq"] * d
    G = case["Hq"] // case["Hkv"]
    return {"bytes": float(lens.sum()) * case["Hkv"] * code + q * (esz + 4), "flops": 4.0 * d * G * case["Hkv"] * float((lens * new).sum())}


# ----------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) + 1)


def _keys_values(g, shape, head_axis, tdt):
    """Keys with a common mean for each head, four strong channels and near-equal norms; values of uneven norms."""
    mean = torch.randn([n if a in (head_axis, 3) else 1 for a, n in enumerate(shape)], device=DEV, generator=g)
    k = torch.randn(shape, device=DEV, generator=g) + 0.35 * mean
    k[..., :4] *= 8.0
    v = torch.randn(shape, device=DEV, generator=g)
    v *= torch.exp(0.5 * torch.randn(shape[:-1] + [1], device=DEV, generator=g))
    return k.to(tdt), v.to(tdt)


def _order(device):
    """Token at each nibble place of a V4 row."""
    p = torch.arange(BLOCK, device=device)
    w, i, e, u, v = p // 16, (p // 8) % 2, (p // 4) % 2, (p // 2) % 2, p % 2
    return 32 * i + 16 * u + 8 * v + 2 * w + e


def prepare(case, seed):
    B, d, op = case["B"], case["d"], case["op"]
    tdt, g = TYPES[case["dtype"]], _gen(seed)
    lens, new = _lens(case, seed)
    s = dict(case=case, lens=torch.tensor(lens, dtype=torch.int64, device=DEV), new=torch.tensor(new, dtype=torch.int64, device=DEV))
    n, H = case["n_max"], case["Hkv"]
    if op == "rope":
        T, Hq = case["T"], case["Hq"]
        # the projections' output: q, k and v of a token side by side
        qkv = (torch.randn(B, T, Hq + 2 * H, d, device=DEV, generator=g) * 1.7).to(tdt)
        s["q"], s["k"], s["v"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + H], qkv[:, :, Hq + H:]
        s["wq"], s["wk"] = [(1 + 0.1 * torch.randn(d, device=DEV, generator=g)).to(tdt) for _ in range(2)]
        inv_freq = 500000.0 ** (-np.arange(0, case["rot"], 2, dtype=np.float64) / case["rot"])
        s["inv_freq"] = torch.tensor(inv_freq, dtype=torch.float64, device=DEV)
        shape = [B, H, n, d] if case["cache"] else [B, T, H, d]
        s["q_out"] = torch.zeros(B, T, Hq, d, device=DEV, dtype=tdt)
        s["K"], s["V"] = torch.zeros(shape, device=DEV, dtype=tdt), torch.zeros(shape, device=DEV, dtype=tdt)
        if own:
            import certified_sparse_attention_gb300 as csa
            s["call"] = csa.QKNormRope(csa.make_shape(B, Hq, H, d, n, case["dtype"]), DEV, wq=s["wq"], wk=s["wk"], norm_eps=1e-6,
                                       inv_freq=inv_freq, interleaved=case["interleaved"])
        return s
    nblk = -(-n // BLOCK)
    k, v = _keys_values(g, [B, H, nblk * BLOCK, d], 1, tdt)
    codes = _quantise(k.view(B, H, nblk, BLOCK, d), v.view(B, H, nblk, BLOCK, d))
    s["K4"], s["bounds"], s["V4"], s["vscale"] = [x.contiguous() for x in codes]
    before = s["lens"] - s["new"] if op == "append" else s["lens"]
    at = (before // BLOCK).clamp(max=nblk - 1).view(B, 1, 1, 1, 1).expand(B, H, 1, BLOCK, d)
    s["Kt"], s["Vt"] = [x.view(B, H, nblk, BLOCK, d).gather(2, at)[:, :, 0].contiguous() for x in (k, v)]
    del k, v
    Hq = case.get("Hq", H)
    if op == "append":
        s["k"], s["v"] = _keys_values(g, [B, case["T"], H, d], 2, tdt)
    if op in ("append", "unpack"):
        rows = case["T"] if op == "append" else case["rows"]
        s["first"] = s["lens"] - s["new"]
        s["K"], s["V"] = [torch.zeros(B, H, rows, d, device=DEV, dtype=tdt) for _ in range(2)]
    else:
        T, G = case["T"], Hq // H
        # half of the heads attend sharply, half almost evenly
        mean = torch.randn(B, 1, H, 1, d, device=DEV, generator=g)
        sharp = torch.where(torch.arange(H, device=DEV) % 2 == 0, 1.0, 0.1).view(1, 1, H, 1, 1)
        q = (0.5 * mean + torch.randn(B, T, H, G, d, device=DEV, generator=g)) * sharp
        s["q"] = q.reshape(B, T, Hq, d).to(tdt)
    if own:
        import certified_sparse_attention_gb300 as csa
        shape = csa.make_shape(B, Hq, H, d, n, case["dtype"])
        s["cache"] = csa.KV4Cache(shape, DEV, buffers=[s[x] for x in ("K4", "bounds", "V4", "vscale", "Kt", "Vt")])
        if op == "decode":
            s["call"] = csa.KV4Decode(shape, DEV, T=case["T"])
    elif op == "decode":
        s["o"] = torch.zeros(B, case["T"], Hq, d, device=DEV)
    return s


# ------------------------------------------------------------------- runs

def run(s):
    op = s["case"]["op"]
    if own:
        if op == "rope":
            s["call"](s["q"], s["k"], s["v"], s["K"], s["V"], s["lens"], s["new"], to_cache=s["case"]["cache"], q_out=s["q_out"])
            return s["q_out"], s["K"], s["V"]
        if op == "append":
            s["cache"].append(s["k"], s["v"], s["lens"], s["new"])
            s["cache"].unpack(s["K"], s["V"], s["lens"], s["first"])
            return s["K"], s["V"], s["Kt"], s["Vt"]
        if op == "unpack":
            s["cache"].unpack(s["K"], s["V"], s["lens"], s["first"])
            return s["K"], s["V"]
        return s["call"](s["q"], s["cache"], s["lens"], s["new"])
    if op == "rope":
        return _rope(s)
    if op == "append":
        _append(s)
        _unpack(s)
        return s["K"], s["V"], s["Kt"], s["Vt"]
    if op == "unpack":
        _unpack(s)
        return s["K"], s["V"]
    return _decode(s)


def _quantise(k, v):
    """Codes and scales of whole blocks [..., 64, d]: K4, bounds, V4, vscale."""
    k, v = k.float(), v.float()
    mn, mx = k.amin(-2, keepdim=True), k.amax(-2, keepdim=True)
    step = (mx - mn) / torch.full_like(mx, 15.0)  # a quotient, where a plain 15 would be a product with 1/15
    step = torch.where(step == 0, torch.ones_like(step), step)
    c = ((k - mn) / step).round_().clamp_(0, 15).to(torch.uint8)
    K4 = c[..., 0::2] | (c[..., 1::2] << 4)
    bounds = torch.cat([mn, step], -2)
    mn, mx = v.amin(-1, keepdim=True), v.amax(-1, keepdim=True)
    step = (mx - mn) / torch.full_like(mx, 15.0)
    c = torch.where(step == 0, torch.zeros_like(v), ((v - mn) / step).round_().clamp_(0, 15)).to(torch.uint8)
    c = c[..., _order(v.device), :].transpose(-1, -2)
    V4 = c[..., 0::2] | (c[..., 1::2] << 4)
    return K4, bounds, V4, torch.cat([mn, step], -1)


def _values(K4, bounds, V4, vscale):
    """What blocks stand for: K and V [..., 64, d] in f32."""
    k = torch.stack([K4 & 15, K4 >> 4], -1).flatten(-2).float()
    k = k * bounds[..., 1:2, :] + bounds[..., 0:1, :]
    c = torch.stack([V4 & 15, V4 >> 4], -1).flatten(-2).transpose(-1, -2)
    back = torch.argsort(_order(V4.device))
    v = c[..., back, :].float() * vscale[..., 1:2] + vscale[..., 0:1]
    return k, v


def _blocks(s):
    """The cache's arrays by block: [B][H][nblk][...]."""
    B, H, d = s["Kt"].shape[0], s["Kt"].shape[1], s["Kt"].shape[3]
    return s["K4"].view(B, H, -1, BLOCK, d // 2), s["bounds"].view(B, H, -1, 2, d), s["V4"].view(B, H, -1, d, BLOCK // 2), \
        s["vscale"].view(B, H, -1, BLOCK, 2)


def _rope(s):
    case = s["case"]
    B, T, rot = case["B"], case["T"], case["rot"]
    start = (s["lens"] - s["new"]).view(B, 1)
    t = torch.arange(T, device=start.device).view(1, T)
    pos, valid = start + t, t < s["new"].view(B, 1)
    angle = pos.double().view(B, T, 1, 1) * s["inv_freq"]
    cos, sin = angle.cos().float(), angle.sin().float()

    def turned(x, w):
        x = x.float()
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()
        y, rest = x[..., :rot], x[..., rot:]
        if case["interleaved"]:
            a, b = y[..., 0::2], y[..., 1::2]
            y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
        else:
            a, b = y[..., :rot // 2], y[..., rot // 2:]
            y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
        return torch.cat([y, rest], -1)

    ok = valid.view(B, T, 1, 1)
    tdt = s["q"].dtype
    s["q_out"].copy_(torch.where(ok, turned(s["q"], s["wq"]).to(tdt), s["q_out"]))
    k = turned(s["k"], s["wk"]).to(tdt)
    if case["cache"]:
        b, t = torch.nonzero(valid, as_tuple=True)
        s["K"][b, :, pos[b, t]] = k[b, t]
        s["V"][b, :, pos[b, t]] = s["v"][b, t]
    else:
        s["K"].copy_(torch.where(ok, k, s["K"]))
        s["V"].copy_(torch.where(ok, s["v"], s["V"]))
    return s["q_out"], s["K"], s["V"]


def _append(s):
    case = s["case"]
    B, T, H, d = case["B"], case["T"], case["Hkv"], case["d"]
    dev = s["lens"].device
    start, n = s["lens"] - s["new"], s["lens"]
    nb = (T + 2 * BLOCK - 2) // BLOCK
    base, r = start // BLOCK, start % BLOCK
    i = torch.arange(nb * BLOCK, device=dev).view(1, -1)
    src = (i - r.view(B, 1)).clamp(0, T - 1)
    old = (i < r.view(B, 1)).view(B, 1, -1, 1)

    def rows(tail, x):
        x = x.gather(1, src.view(B, -1, 1, 1).expand(B, nb * BLOCK, H, d)).transpose(1, 2)
        return torch.where(old, tail.repeat(1, 1, nb, 1), x)

    k, v = rows(s["Kt"], s["k"]), rows(s["Vt"], s["v"])
    j = torch.arange(nb, device=dev).view(1, nb)
    blk = base.view(B, 1) + j
    done = (blk + 1) * BLOCK <= n.view(B, 1)
    b = torch.arange(B, device=dev).view(B, 1)
    fresh = _quantise(k.view(B, H, nb, BLOCK, d), v.view(B, H, nb, BLOCK, d))
    at = blk.clamp(max=s["bounds"].shape[2] - 1)

    def put(into, x):
        x = x.transpose(1, 2)
        into[b, :, at] = torch.where(done.view(B, nb, 1, 1, 1), x, into[b, :, at])

    [put(a, x) for a, x in zip(_blocks(s), fresh)]
    # the rows of the incomplete block
    p = torch.arange(BLOCK, device=dev).view(1, BLOCK)
    keep = (p < (n % BLOCK).view(B, 1)).view(B, 1, BLOCK, 1)
    last = ((n // BLOCK - base).view(B, 1) * BLOCK + p).clamp(max=nb * BLOCK - 1).view(B, 1, BLOCK, 1).expand(B, H, BLOCK, d)
    s["Kt"].copy_(torch.where(keep, k.gather(2, last), s["Kt"]))
    s["Vt"].copy_(torch.where(keep, v.gather(2, last), s["Vt"]))


def _unpack(s):
    B, H, rows, d = s["K"].shape
    dev = s["lens"].device
    first, n = s["first"], s["lens"]
    nb = (rows + 2 * BLOCK - 2) // BLOCK
    base = first // BLOCK
    b = torch.arange(B, device=dev).view(B, 1)
    at = (base.view(B, 1) + torch.arange(nb, device=dev)).clamp(max=s["bounds"].shape[2] - 1)
    k, v = _values(*[x[b, :, at] for x in _blocks(s)])
    pos = first.view(B, 1) + torch.arange(rows, device=dev)
    src = (pos - base.view(B, 1) * BLOCK)
    tail = (pos // BLOCK >= (n // BLOCK).view(B, 1)).view(B, 1, rows, 1)
    ok = (pos < n.view(B, 1)).view(B, 1, rows, 1)

    def out(x, t, into):
        x = x.transpose(1, 2).reshape(B, H, nb * BLOCK, d).gather(2, src.view(B, 1, rows, 1).expand(B, H, rows, d))
        t = t.gather(2, (pos % BLOCK).view(B, 1, rows, 1).expand(B, H, rows, d))
        into.copy_(torch.where(ok, torch.where(tail, t, x.to(t.dtype)), into))

    out(k, s["Kt"], s["K"])
    out(v, s["Vt"], s["V"])


def _decode(s):
    case = s["case"]
    B, T, H, d = case["B"], case["T"], case["Hkv"], case["d"]
    G, n, dev = case["Hq"] // H, s["lens"], s["lens"].device
    k, v = _values(*_blocks(s))
    nblk = k.shape[2]
    whole = (torch.arange(nblk, device=dev) < (n // BLOCK).view(B, 1)).view(B, 1, nblk, 1, 1)
    k = torch.where(whole, k, s["Kt"].float().unsqueeze(2)).flatten(2, 3)
    v = torch.where(whole, v, s["Vt"].float().unsqueeze(2)).flatten(2, 3)
    q = s["q"].float().view(B, T, H, G, d).permute(0, 2, 1, 3, 4).reshape(B, H, T * G, d)
    score = torch.matmul(q, k.transpose(2, 3)) / math.sqrt(d)
    t = torch.arange(T, device=dev)
    end = n.view(B, 1) - s["new"].view(B, 1) + t  # last position each row attends to
    seen = torch.arange(nblk * BLOCK, device=dev) <= end.view(B, 1, T, 1, 1)
    score = torch.where(seen, score.view(B, H, T, G, -1), torch.full_like(score[:1, :1, :1, :1], -math.inf))
    p = torch.exp(score - score.amax(-1, keepdim=True))
    p = (p / p.sum(-1, keepdim=True)).view(B, H, T * G, nblk, BLOCK)
    o = torch.matmul(p.transpose(2, 3), v.view(B, H, nblk, BLOCK, d)).sum(2)  # a product for each block, then their sum
    o = o.view(B, H, T, G, d).transpose(1, 2).reshape(B, T, H * G, d)
    s["o"].copy_(torch.where((t < s["new"].view(B, 1)).view(B, T, 1, 1), o, s["o"]))
    return s["o"]


# ------------------------------------------------- definitions in 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"rope": _exact_rope, "append": _exact_append, "unpack": _exact_unpack, "decode": _exact_decode}[case["op"]](s)


def _exact_rope(s):
    case = s["case"]
    rot, half = case["rot"], case["rot"] // 2
    q_out, K, V = s["q_out"].double(), s["K"].double(), s["V"].double()
    lo = np.arange(half) * 2 if case["interleaved"] else np.arange(half)
    hi = lo + 1 if case["interleaved"] else lo + half
    lo, hi = torch.tensor(lo, device=DEV), torch.tensor(hi, device=DEV)
    for b in range(case["B"]):
        m, n = int(s["new"][b]), int(s["lens"][b])
        pos = torch.arange(n - m, n, device=DEV, dtype=torch.float64)
        z = torch.polar(torch.ones(m, half, device=DEV, dtype=torch.float64), pos[:, None] * s["inv_freq"][None])[:, None]
        for x, w, kind in ((s["q"], s["wq"], "q"), (s["k"], s["wk"], "k")):
            x = x[b, :m].double()
            x = x / ((x * x).sum(-1, keepdim=True) / x.shape[-1] + 1e-6).sqrt() * w.double()
            pair = torch.complex(x[..., lo], x[..., hi]) * z
            x[..., lo], x[..., hi] = pair.real, pair.imag
            if kind == "q":
                q_out[b, :m] = x
            elif case["cache"]:
                K[b, :, n - m:n] = x.transpose(0, 1)
                V[b, :, n - m:n] = s["v"][b, :m].double().transpose(0, 1)
            else:
                K[b, :m], V[b, :m] = x, s["v"][b, :m].double()
    return q_out, K, V


def _f32(x):
    """A rounding to 32 bits that the definition of the codes names: it decides values half way between two codes."""
    return x.float().double()


def _nibbles(x):
    return torch.stack([x & 15, x >> 4], -1).flatten(-2).double()


def _place():
    t = np.arange(BLOCK)
    return torch.tensor(16 * ((t // 2) % 4) + 8 * (t // 32) + 4 * (t % 2) + 2 * ((t // 16) % 2) + (t // 8) % 2, device=DEV)


def _exact_rows(s, b, lo, hi, n):
    """Rows [lo, hi) of sequence b's cache of n tokens, [H][hi - lo][d] in 64 bits."""
    H, d = s["Kt"].shape[1], s["Kt"].shape[3]
    first, last = lo // BLOCK, min(-(-hi // BLOCK), n // BLOCK)
    bd, vs = s["bounds"][b, :, first:last].double(), s["vscale"].view(s["Kt"].shape[0], H, -1, BLOCK, 2)[b, :, first:last].double()
    K4, V4 = [x.view(s["Kt"].shape[0], H, -1, *shape)[b, :, first:last] for x, shape in ((s["K4"], (BLOCK, d // 2)), (s["V4"], (d, BLOCK // 2)))]
    k = (bd[:, :, :1] + _nibbles(K4) * bd[:, :, 1:]).reshape(H, -1, d)
    v = (vs[..., :1] + _nibbles(V4)[..., _place()].transpose(-1, -2) * vs[..., 1:]).reshape(H, -1, d)
    k, v = [torch.cat([x, t[b, :, :n % BLOCK].double()], 1) if hi > n // BLOCK * BLOCK else x for x, t in ((k, s["Kt"]), (v, s["Vt"]))]
    return [x[:, lo - first * BLOCK:hi - first * BLOCK] for x in (k, v)]


def _exact_unpack(s):
    K, V = s["K"].double(), s["V"].double()
    for b in range(K.shape[0]):
        lo, n = int(s["first"][b]), int(s["lens"][b])
        hi = min(n, lo + K.shape[2])
        K[b, :, :hi - lo], V[b, :, :hi - lo] = _exact_rows(s, b, lo, hi, n)
    return K, V


def _exact_append(s):
    K, V, Kt, Vt = [s[x].double() for x in ("K", "V", "Kt", "Vt")]
    for b in range(K.shape[0]):
        m, n = int(s["new"][b]), int(s["lens"][b])
        r, whole = (n - m) % BLOCK, n // BLOCK * BLOCK
        base = n - m - r
        for new, tail, rows, per_token in ((s["k"], Kt, K, False), (s["v"], Vt, V, True)):
            x = torch.cat([tail[b, :, :r].clone(), new[b, :m].double().transpose(0, 1)], 1)
            y = x[:, :whole - base].reshape(x.shape[0], -1, BLOCK, x.shape[2])
            left = x[:, max(0, whole - base):]
            if y.numel():
                axis = 3 if per_token else 2
                lo, up = y.min(axis, keepdim=True).values, y.max(axis, keepdim=True).values
                step = _f32(_f32(up - lo) / 15)
                y = lo + step * torch.round(_f32(_f32(y - lo) / torch.where(step == 0, 1.0, step)))
            x = torch.cat([y.reshape(x.shape[0], -1, x.shape[2]), left], 1)
            rows[b, :, :m] = x[:, r:]
            if n % BLOCK:
                tail[b, :, :n % BLOCK] = left
    return K, V, Kt, Vt


def _exact_decode(s):
    case = s["case"]
    G, H, d = case["Hq"] // case["Hkv"], case["Hkv"], case["d"]
    o = s["o"].double()
    for b in range(case["B"]):
        n, m = int(s["lens"][b]), int(s["new"][b])
        k, v = _exact_rows(s, b, 0, n, n)
        for t in range(m):
            e = n - m + t + 1
            q = s["q"][b, t].double().view(H, G, d)
            score = q @ k[:, :e].transpose(1, 2) / math.sqrt(d)
            o[b, t] = (torch.softmax(score, -1) @ v[:, :e]).reshape(H * G, d)
    return o
