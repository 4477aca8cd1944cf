"""Cases that measure the K/V cache held in 8 bits: its append (``csa_kv8_append``), reading it back (``csa_kv8_unpack``), the
attention over all of it (``csa_kv8_decode``), the choice of blocks by a cheap score (``csa_kv8_select``) and the attention over
the chosen blocks (``csa_kv8_decode_blocks``).

With ``own`` false, ``run`` computes an operator from elementary torch operations; with ``own`` true it makes the calls a user
makes of the library.  Lengths live on the device, as in a decode loop replayed from a CUDA graph.

The 8-bit cache of one (sequence, KV head), in blocks of 64 tokens.  Codes -127 .. 127 are held plus 128:
  K8      [8][d/64][8][64] per block: element (j, h, g, c) is token 16 (g / 2) + 2 j + g % 2, channel 64 h + c
  V8      [d][64] per block: row = channel
  scale   [2] per block: the step of its keys, that of its values (largest magnitude / 127)
  span    [2][d] per block: each channel's largest and smallest key code
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
        # one decode step's new tokens into the cache, and the block that holds each read back
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
        # several drafted tokens of each sequence checked at once, f32, small heads
        dict(name="decode drafts f32", op="decode", B=8, T=5, Hq=32, Hkv=8, d=64, dtype="f32", n_max=30001, ragged=True),
        # the benchmark's step: 128K tokens, four sequences, 32/8 heads
        dict(name="decode long", op="decode", B=4, T=1, Hq=32, Hkv=8, d=128, dtype="bf16", n_max=131072, ragged=False),
        # the choice alone, for a batch of uneven lengths
        dict(name="select batch", op="select", B=64, T=1, Hq=32, Hkv=8, d=128, dtype="bf16", n_max=16000, ragged=True,
             n_sel=16, n_first=1, n_last=2),
        # ... and in one context of a million tokens
        dict(name="select far", op="select", B=1, T=1, Hq=32, Hkv=8, d=128, dtype="bf16", n_max=1048576, ragged=False,
             n_sel=256, n_first=1, n_last=4),
        # the benchmark's step on 64 of its 2048 blocks: choice and attention
        dict(name="sparse long", op="sparse", B=4, T=1, Hq=32, Hkv=8, d=128, dtype="bf16", n_max=131072, ragged=False,
             n_sel=64, n_first=1, n_last=2),
        # drafted tokens, each with blocks of its own, in a batch of uneven lengths
        dict(name="sparse drafts", op="sparse", B=24, T=4, Hq=32, Hkv=8, d=128, dtype="bf16", n_max=30000, ragged=True,
             n_sel=40, n_first=1, n_last=2),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["append", "unpack", "decode", "decode", "select", "sparse", "sparse"])
    d, dtype = rng.choice([64, 128]), rng.choice(["bf16", "bf16", "f32"])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    Hq = Hkv * rng.choice([1, 2, 4, 8])
    B = _log(rng, 1, 64)
    ragged = rng.random() < 0.75
    if op == "append":
        T = _log(rng, 1, max(1, min(8191, (1 << 17) // (B * Hkv))))
        return dict(op=op, B=B, T=T, Hkv=Hkv, d=d, dtype=dtype, n_max=T + 128 + _log(rng, 1, 2048), ragged=ragged)
    if op == "unpack":
        rows = _log(rng, 1, max(1, min(32768, (1 << 19) // (B * Hkv))))
        return dict(op=op, B=B, rows=rows, Hkv=Hkv, d=d, dtype=dtype, n_max=rows + _log(rng, 1, 512), ragged=ragged)
    T = min(rng.choice([1, 1, 1, 2, 3, 5, 8, 16]), 64 // (Hq // Hkv))
    n = _log(rng, 1, max(1, min(131072, (1 << 21) // (B * Hkv))))
    case = dict(op=op, B=B, T=T, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, n_max=n, ragged=ragged)
    if op == "decode":
        return case
    first, last = rng.choice([0, 1, 1, 2]), rng.choice([1, 2, 2, 4])
    sel = first + last + _log(rng, 1, max(1, min(128, (1 << 15) // (B * Hkv * T)))) - 1
    return dict(case, n_sel=sel, n_first=first, n_last=last)


def _lens(case, seed):
    """Lengths of the sequences after this pass's new tokens, and how many of those there are, on the host."""
    r = np.random.RandomState(seed % (1 << 31))
    B, n = case["B"], case["n_max"]
    if case["op"] in ("append", "unpack"):
        rows = case["T"] if case["op"] == "append" else case["rows"]
        new = r.randint(rows // 2 + 1, rows + 1, B) if case["ragged"] else np.full(B, rows)
        new[0] = rows
        # room for the block-aligned rows around the new ones
        top = n - 2 * BLOCK if case["op"] == "append" else n
        return new + r.randint(0, max(1, top - rows + 1), B), new
    lens = r.randint(n // 8 + 1, n + 1, B) if case["ragged"] else np.full(B, n)
    lens[0] = n
    new = np.minimum(lens, r.randint(1, case["T"] + 1, B) if case["ragged"] else case["T"])
    return lens, new


def work(case):
    B, d, esz = case["B"], case["d"], 2 if case["dtype"] == "bf16" else 4
    lens, new = _lens(case, 7)
    op, H = case["op"], case["Hkv"]
    code = 2 * d + 8 / BLOCK         # bytes of one token of one KV head: codes, steps
    span = 2 * d + 4                 # bytes a block's score needs: spans, the keys' step
    rows = float(new.sum()) * H
    if op == "append":  # rows in, codes out (full precision while their block is incomplete), rows read back
        if case["T"] == 1:
            return {"bytes": rows * 6 * d * esz, "flops": 0}
        return {"bytes": rows * (4 * d * esz + 2 * code + 2 * d / BLOCK), "flops": 12.0 * d * rows}
    if op == "unpack":
        return {"bytes": rows * (2 * d * esz + code), "flops": 4.0 * d * rows}
    q, G = float(new.sum()) * case["Hq"] * d, case["Hq"] // H
    whole = lens // BLOCK
    if op == "decode":
        return {"bytes": float(lens.sum()) * H * code + q * (esz + 4), "flops": 4.0 * d * G * H * float((lens * new).sum())}
    sel = np.minimum(-(-lens // BLOCK), case["n_sel"])
    ids = float((new * sel).sum()) * H
    out = {"bytes": float(whole.sum()) * H * span + q * esz + 4.0 * ids, "flops": 4.0 * d * G * H * float((whole * new).sum())}
    if op == "sparse":
        # a block that several tokens of a sequence choose is read once
        out["bytes"] += float(np.minimum(new * sel, -(-lens // BLOCK)).sum()) * H * BLOCK * code + q * 4
        out["flops"] += 4.0 * d * G * BLOCK * ids
    return out


# ----------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) + 1)


def _keys_values(g, shape, head_axis, tdt):
    """Keys with a common mean for each head, four strong channels and near-equal norms; values of uneven norms."""
    mean = torch.randn([n if a in (head_axis, 3) else 1 for a, n in enumerate(shape)], device=DEV, generator=g)
    k = torch.randn(shape, device=DEV, generator=g).add_(0.35 * mean)
    k[..., :4] *= 8.0
    v = torch.randn(shape, device=DEV, generator=g)
    v *= torch.exp(0.5 * torch.randn(shape[:-1] + [1], device=DEV, generator=g))
    return k.to(tdt), v.to(tdt)


def prepare(case, seed):
    B, d, op, H, n = case["B"], case["d"], case["op"], case["Hkv"], case["n_max"]
    tdt, g = TYPES[case["dtype"]], _gen(seed)
    lens, new = _lens(case, seed)
    s = dict(case=case, lens=torch.tensor(lens, dtype=torch.int64, device=DEV), new=torch.tensor(new, dtype=torch.int64, device=DEV))
    nblk = -(-n // BLOCK)
    k, v = _keys_values(g, [B, H, nblk * BLOCK, d], 1, tdt)
    if op in ("select", "sparse"):
        # neighbouring tokens are alike: a drift of each block
        k += torch.randn(B, H, nblk, 1, d, device=DEV, generator=g).expand(B, H, nblk, BLOCK, d).reshape(k.shape).to(tdt)
    codes = [torch.cat(x, 2) for x in zip(*[_quantise(k[:, :, i:i + (1 << 17)].reshape(B, H, -1, BLOCK, d),
                                                      v[:, :, i:i + (1 << 17)].reshape(B, H, -1, BLOCK, d))
                                            for i in range(0, nblk * BLOCK, 1 << 17)])]
    s["K8"], s["V8"], s["scale"], s["span"] = [x.contiguous() for x in codes]
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
        s["cache"] = csa.KV8Cache(shape, DEV, buffers=[s[x] for x in ("K8", "V8", "scale", "span", "Kt", "Vt")])
        if op == "decode":
            s["call"] = csa.KV8Decode(shape, DEV, T=case["T"])
        elif op in ("select", "sparse"):
            s["call"] = csa.KV8Sparse(shape, DEV, case["n_sel"], T=case["T"], n_first=case["n_first"], n_last=case["n_last"])
    elif op in ("decode", "sparse"):
        s["o"] = torch.zeros(B, case["T"], Hq, d, device=DEV)
    if op in ("select", "sparse") and not own:
        s["blocks"] = torch.zeros(B, case["T"], H, case["n_sel"], device=DEV, dtype=torch.int32)
        s["count"] = torch.zeros(B, case["T"], H, device=DEV, dtype=torch.int32)
    return s


# ------------------------------------------------------------------- runs

def run(s):
    op = s["case"]["op"]
    if own:
        if op == "append":
            s["cache"].append(s["k"], s["v"], s["lens"], s["new"])
            s["cache"].unpack(s["K"], s["V"], s["lens"], s["first"])
            return s["K"], s["V"], s["Kt"], s["Vt"], s["span"]
        if op == "unpack":
            s["cache"].unpack(s["K"], s["V"], s["lens"], s["first"])
            return s["K"], s["V"]
        if op == "decode":
            return s["call"](s["q"], s["cache"], s["lens"], s["new"])
        if op == "select":
            return s["call"].select(s["q"], s["cache"], s["lens"], s["new"])
        o = s["call"](s["q"], s["cache"], s["lens"], s["new"])
        return o, s["call"].blocks, s["call"].count
    if op == "append":
        _append(s)
        _unpack(s)
        return s["K"], s["V"], s["Kt"], s["Vt"], s["span"]
    if op == "unpack":
        _unpack(s)
        return s["K"], s["V"]
    if op == "decode":
        return _decode(s)
    _select(s)
    if op == "select":
        return s["blocks"], s["count"]
    return _attend(s), s["blocks"], s["count"]


def _coded(c):
    """Whole numbers -127 .. 127 as the cache holds them."""
    return (c + 128).to(torch.uint8)


def _number(code):
    """... and back, in f32."""
    return code.float() - 128


def _step(top):
    step = top / torch.full_like(top, 127.0)  # a quotient, where a plain 127 would be a product with 1/127
    return torch.where(step == 0, torch.ones_like(step), step)


def _keys_in_order(c):
    """Keys [..., 64, d] in K8's order: [..., 8, d/64, 8, 64]."""
    c = c.unflatten(-2, (4, 8, 2)).unflatten(-1, (-1, 64))
    n = c.dim() - 5
    return c.permute(*range(n), n + 1, n + 3, n, n + 2, n + 4).flatten(-3, -2)


def _keys_back(c):
    c = c.unflatten(-2, (4, 2))
    n = c.dim() - 5
    return c.permute(*range(n), n + 2, n, n + 3, n + 1, n + 4).flatten(-5, -3).flatten(-2)


def _quantise(k, v):
    """Codes, steps and spans of whole blocks [..., 64, d]: K8, V8, scale, span."""
    k, v = k.float(), v.float()
    sk, sv = [_step(x.abs().amax((-2, -1), keepdim=True)) for x in (k, v)]
    ck, cv = [(x / s).round_().clamp_(-127, 127).nan_to_num_(0) for x, s in ((k, sk), (v, sv))]
    span = torch.stack([ck.amax(-2), ck.amin(-2)], -2)
    return _coded(_keys_in_order(ck)), _coded(cv.transpose(-1, -2)), torch.cat([sk, sv], -1)[..., 0, :], _coded(span)


def _values(K8, V8, scale):
    """What blocks stand for: K and V [..., 64, d] in f32."""
    k = _keys_back(_number(K8)) * scale[..., 0, None, None]
    return k, _number(V8).transpose(-1, -2) * scale[..., 1, None, None]


def _blocks(s):
    """The cache's arrays by block: [B][H][nblk][...]."""
    B, H, d = s["Kt"].shape[0], s["Kt"].shape[1], s["Kt"].shape[3]
    return s["K8"].view(B, H, -1, 8, d // 64, 8, 64), s["V8"].view(B, H, -1, d, BLOCK), s["scale"].view(B, H, -1, 2), \
        s["span"].view(B, H, -1, 2, d)


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
    fresh = _quantise(k.reshape(B, H, nb, BLOCK, d), v.reshape(B, H, nb, BLOCK, d))
    at = blk.clamp(max=s["scale"].shape[2] - 1)

    def put(into, x):
        x = x.transpose(1, 2)
        into[b, :, at] = torch.where(done.view([B, nb] + [1] * (x.dim() - 2)), x, into[b, :, at])

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
    at = (base.view(B, 1) + torch.arange(nb, device=dev)).clamp(max=s["scale"].shape[2] - 1)
    k, v = _values(*[x[b, :, at] for x in _blocks(s)[:3]])
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


def _softmax(score):
    p = torch.exp(score - score.amax(-1, keepdim=True))
    return p / p.sum(-1, keepdim=True)


def _decode(s):
    case = s["case"]
    B, T, H, d = case["B"], case["T"], case["Hkv"], case["d"]
    G, n, dev = case["Hq"] // H, s["lens"], s["lens"].device
    k, v = _values(*_blocks(s)[:3])
    nblk = k.shape[2]
    whole = (torch.arange(nblk, device=dev) < (n // BLOCK).view(B, 1)).view(B, 1, nblk, 1, 1)
    k = torch.where(whole, k, s["Kt"].float().unsqueeze(2)).flatten(2, 3)
    v = torch.where(whole, v, s["Vt"].float().unsqueeze(2)).flatten(2, 3)
    q = s["q"].float().view(B, T, H, G, d).permute(0, 2, 1, 3, 4).reshape(B, H, T * G, d)
    score = torch.matmul(q, k.transpose(2, 3)) / math.sqrt(d)
    t = torch.arange(T, device=dev)
    end = n.view(B, 1) - s["new"].view(B, 1) + t  # last position each row attends to
    seen = torch.arange(nblk * BLOCK, device=dev) <= end.clamp(min=0).view(B, 1, T, 1, 1)
    score = score.view(B, H, T, G, -1).masked_fill(~seen, -math.inf)
    p = _softmax(score).view(B, H, T * G, nblk, BLOCK)
    o = torch.matmul(p.transpose(2, 3), v.view(B, H, nblk, BLOCK, d)).sum(2)  # a product for each block, then their sum
    o = o.view(B, H, T, G, d).transpose(1, 2).reshape(B, T, H * G, d)
    s["o"].copy_(torch.where((t < s["new"].view(B, 1)).view(B, T, 1, 1), o, s["o"]))
    return s["o"]


def _select(s):
    """The blocks of each token and KV head.  A block's score: the query head rounded to 8 bits, against the end of each
    channel's span that its sign asks for; the largest over the heads."""
    case = s["case"]
    B, T, H, d, N = case["B"], case["T"], case["Hkv"], case["d"], case["n_sel"]
    G, dev = case["Hq"] // H, s["lens"].device
    q = s["q"].float().view(B, T, H, G, d)
    step = _step(q.abs().amax(-1, keepdim=True))
    c = (q / step).round_().clamp_(-127, 127).nan_to_num_(0).permute(0, 2, 1, 3, 4).reshape(B, H, T * G, d)
    span = _number(_blocks(s)[3])
    # whole numbers below 2^24: exact in any order
    dots = torch.matmul(c.clamp(min=0), span[:, :, :, 0].transpose(2, 3)) + torch.matmul(c.clamp(max=0), span[:, :, :, 1].transpose(2, 3))
    score = (dots.view(B, H, T, G, -1) * _blocks(s)[2][:, :, None, None, :, 0]) * step.squeeze(-1).permute(0, 2, 1, 3).unsqueeze(-1)
    score = score.amax(3).double().nan_to_num_(1e300, 1e300).transpose(1, 2)       # [B][T][H][nblk]
    nblk = score.shape[-1]
    t = torch.arange(T, device=dev)
    mine = ((s["lens"] - s["new"]).view(B, 1) + t).view(B, T, 1, 1) // BLOCK       # the token's own block
    j = torch.arange(nblk, device=dev)
    score = torch.where((j < case["n_first"]) | (j > mine - case["n_last"]), math.inf, score)
    score = torch.where(j > mine, -math.inf, score)
    best = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :N]
    count = (mine + 1).clamp(max=N)
    best = torch.where(torch.arange(best.shape[-1], device=dev) < count, best, nblk)
    best = torch.sort(best, dim=-1).values
    best = torch.where(best == nblk, -1, best).int()
    if best.shape[-1] < N:
        best = torch.cat([best, torch.full([B, T, H, N - best.shape[-1]], -1, device=dev, dtype=torch.int32)], -1)
    ok = (t < s["new"].view(B, 1)).view(B, T, 1, 1)
    s["blocks"].copy_(torch.where(ok, best, s["blocks"]))
    s["count"].copy_(torch.where(ok[..., 0], count[..., 0].int(), s["count"]))


def _attend(s):
    case = s["case"]
    B, T, H, d, N = case["B"], case["T"], case["Hkv"], case["d"], case["n_sel"]
    G, n, dev = case["Hq"] // H, s["lens"], s["lens"].device
    ids = s["blocks"].long()
    K8, V8, scale, _ = _blocks(s)
    b = torch.arange(B, device=dev).view(B, 1, 1, 1)
    h = torch.arange(H, device=dev).view(1, 1, H, 1)
    at = ids.clamp(0, K8.shape[2] - 1)
    k, v = _values(K8[b, h, at], V8[b, h, at], scale[b, h, at])                    # [B][T][H][N][64][d]
    tail = (ids == (n // BLOCK).view(B, 1, 1, 1))[..., None, None]
    k = torch.where(tail, s["Kt"].float()[:, None, :, None], k).flatten(3, 4)
    v = torch.where(tail, s["Vt"].float()[:, None, :, None], v)
    q = s["q"].float().view(B, T, H, G, d)
    score = torch.matmul(q, k.transpose(3, 4)) / math.sqrt(d)                      # [B][T][H][G][N * 64]
    t = torch.arange(T, device=dev)
    end = (n.view(B, 1) - s["new"].view(B, 1) + t).view(B, T, 1, 1, 1)
    pos = ids[..., None] * BLOCK + torch.arange(BLOCK, device=dev)
    listed = torch.arange(N, device=dev) < s["count"][..., None]
    seen = (listed[..., None] & (pos <= end)).flatten(3).unsqueeze(3)
    p = _softmax(score.masked_fill(~seen, -math.inf)).view(B, T, H, G, N, BLOCK)
    o = torch.matmul(p.transpose(3, 4), v).sum(3).reshape(B, T, H * G, d)
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
    return {"append": _exact_append, "unpack": _exact_unpack, "decode": _exact_decode, "select": _exact_select,
            "sparse": _exact_sparse}[case["op"]](s)


def _f32(x):
    """A rounding to 32 bits that the definition of the codes names: it decides values half way between two codes."""
    return x.float().double()


def _place(d):
    """Where K8 holds (token, channel), as an index into the flat block."""
    t, c = np.arange(BLOCK)[:, None], np.arange(d)[None]
    return torch.tensor(((t % 16 // 2 * (d // 64) + c // 64) * 8 + t // 16 * 2 + t % 2) * 64 + c % 64, device=DEV)


def _signed(code):
    return (code.long() - 128).double()


def _exact_block(s, b, h, j):
    """Keys and values [len(j)][64][d] that whole blocks j of (b, h) stand for."""
    B, H, d = s["Kt"].shape[0], s["Kt"].shape[1], s["Kt"].shape[3]
    K8, V8, scale = s["K8"].view(B, H, -1, BLOCK * d)[b, h], s["V8"].view(B, H, -1, d, BLOCK)[b, h], s["scale"].view(B, H, -1, 2)[b, h]
    k = _signed(K8[j][:, _place(d)]) * scale[j, :1, None].double()
    return k, _signed(V8[j]).transpose(1, 2) * scale[j, 1:, None].double()


def _exact_rows(s, b, h, lo, hi, n):
    """Rows [lo, hi) of the cache of (b, h), n tokens long."""
    first, last = lo // BLOCK, min(-(-hi // BLOCK), n // BLOCK)
    k, v = [x.flatten(0, 1) for x in _exact_block(s, b, h, torch.arange(first, max(first, last), device=DEV))]
    if hi > n // BLOCK * BLOCK:
        k, v = torch.cat([k, s["Kt"][b, h, :n % BLOCK].double()]), torch.cat([v, s["Vt"][b, h, :n % BLOCK].double()])
    return k[lo - first * BLOCK:hi - first * BLOCK], v[lo - first * BLOCK:hi - first * BLOCK]


def _exact_unpack(s):
    K, V = s["K"].double(), s["V"].double()
    for b in range(K.shape[0]):
        lo, n = int(s["first"][b]), int(s["lens"][b])
        hi = min(n, lo + K.shape[2])
        for h in range(K.shape[1]):
            K[b, h, :hi - lo], V[b, h, :hi - lo] = _exact_rows(s, b, h, lo, hi, n)
    return K, V


def _exact_append(s):
    K, V, Kt, Vt = [s[x].double() for x in ("K", "V", "Kt", "Vt")]
    B, H, d = Kt.shape[0], Kt.shape[1], Kt.shape[3]
    span = s["span"].clone()
    flat = span.view(B, H, -1, 2, d)
    for b in range(B):
        m, n = int(s["new"][b]), int(s["lens"][b])
        r, whole = (n - m) % BLOCK, n // BLOCK * BLOCK
        base = n - m - r
        for new, tail, rows in ((s["k"], Kt, K), (s["v"], Vt, V)):
            x = torch.cat([tail[b, :, :r].clone(), new[b, :m].double().transpose(0, 1)], 1)
            y = x[:, :max(0, whole - base)].reshape(H, -1, BLOCK, d)
            left = x[:, max(0, whole - base):]
            if y.numel():
                step = _f32(torch.maximum(y.amax((2, 3), keepdim=True), -y.amin((2, 3), keepdim=True)) / 127)
                step = torch.where(step == 0, 1.0, step)
                c = torch.round(_f32(y / step)).clamp(-127, 127)
                y = c * step
                if new is s["k"]:
                    ends = torch.stack([c.max(2).values, c.min(2).values], 2)
                    flat[b, :, base // BLOCK:whole // BLOCK] = (ends + 128).to(torch.uint8)
            x = torch.cat([y.reshape(H, -1, d), left], 1)
            rows[b, :, :m] = x[:, r:]
            if n % BLOCK:
                keep = n % BLOCK
                tail[b, :, :keep] = x[:, x.shape[1] - keep:]
    return K, V, Kt, Vt, span


def _exact_decode(s):
    case = s["case"]
    G, H, d = case["Hq"] // case["Hkv"], case["Hkv"], case["d"]
    o = s["o"].double()
    for b in range(case["B"]):
        n, m = int(s["lens"][b]), int(s["new"][b])
        for h in range(H):
            k, v = _exact_rows(s, b, h, 0, n, n)
            for t in range(m):
                e = n - m + t + 1
                score = s["q"][b, t, h * G:(h + 1) * G].double() @ k[:e].T / math.sqrt(d)
                o[b, t, h * G:(h + 1) * G] = torch.softmax(score, -1) @ v[:e]
    return o


def _exact_choice(s):
    """Lists of blocks, scored in whole numbers and the two roundings that the definition of the score names."""
    case = s["case"]
    B, T, H, d, N = case["B"], case["T"], case["Hkv"], case["d"], case["n_sel"]
    G = case["Hq"] // H
    blocks, count = s["blocks"].clone(), s["count"].clone()
    span, scale = s["span"].view(B, H, -1, 2, d), s["scale"].view(B, H, -1, 2)
    for b in range(B):
        n, m = int(s["lens"][b]), int(s["new"][b])
        for t in range(m):
            o = (n - m + t) // BLOCK
            q = s["q"][b, t].double().view(H, G, d)
            step = _f32(q.abs().max(-1, keepdim=True).values / 127)
            step = torch.where(step == 0, 1.0, step)
            c = torch.round(_f32(q / step)).clamp(-127, 127)[:, :, None]                    # [H][G][1][d]
            ends = _signed(span[b, :, :o + 1])[:, None]                                     # [H][1][o + 1][2][d]
            dots = torch.stack([torch.maximum(c[:, i] * ends[:, 0, :, 0], c[:, i] * ends[:, 0, :, 1]).sum(-1) for i in range(G)], 1)
            score = _f32(_f32(dots * scale[b, :, None, :o + 1, 0].double()) * step).max(1).values.cpu().numpy()
            for h in range(H):
                kept = set(range(o + 1)) if o + 1 <= N else \
                    set(range(case["n_first"])) | set(range(o + 1 - case["n_last"], o + 1))
                order = np.lexsort((np.arange(o + 1), -score[h]))
                for x in order:
                    if len(kept) >= min(N, o + 1):
                        break
                    kept.add(int(x))
                row = sorted(kept)
                blocks[b, t, h] = torch.tensor(row + [-1] * (N - len(row)), dtype=torch.int32)
                count[b, t, h] = len(row)
    return blocks, count


def _exact_select(s):
    return _exact_choice(s)


def _exact_sparse(s):
    case = s["case"]
    G, H, d = case["Hq"] // case["Hkv"], case["Hkv"], case["d"]
    blocks, count = _exact_choice(s)
    o = s["o"].double()
    for b in range(case["B"]):
        n, m = int(s["lens"][b]), int(s["new"][b])
        for t in range(m):
            e = n - m + t + 1
            for h in range(H):
                ids = blocks[b, t, h, :int(count[b, t, h])].long()
                ids = ids[ids < n // BLOCK]
                k, v = [x.flatten(0, 1) for x in _exact_block(s, b, h, ids)]
                pos = (ids[:, None] * BLOCK + torch.arange(BLOCK, device=DEV)).flatten()
                if (e - 1) // BLOCK == n // BLOCK:
                    left = n % BLOCK
                    k, v = torch.cat([k, s["Kt"][b, h, :left].double()]), torch.cat([v, s["Vt"][b, h, :left].double()])
                    pos = torch.cat([pos, n // BLOCK * BLOCK + torch.arange(left, device=DEV)])
                score = s["q"][b, t, h * G:(h + 1) * G].double() @ k.T / math.sqrt(d)
                score = score.masked_fill(pos >= e, -math.inf)
                o[b, t, h * G:(h + 1) * G] = torch.softmax(score, -1) @ v
    return o, blocks, count
