"""Operators of a paged KV cache held in 4 bits, in plain torch and as this framework's calls.

  store   RoPE of the new rows, quantised as they are written into the cache, and the rows read
          back as the cache now holds them
  read    cached tokens of a batch of sequences as contiguous bf16 rows
  decode  single-token attention over the cache
  step    the fused decode step: rotate, quantise and store each sequence's new token, then attend
          (and the token's row as the cache holds it)
  prefill causal attention of a chunk's queries over everything cached

Common shapes: head_dim 128, 16-token blocks, block tables [sequences][max_blocks] int32.  The cache is
uint8 [num_blocks][kv_heads][2208]; a record holds one (block, KV head):

  0     K codes, 64 bytes a token: the 32-bit word of dims 32 g + 8 i .. + 7 is word 4 i + g of the
        token's sixteen
  1024  V codes, 64 bytes a token: dims 32 u .. 32 u + 31 are its 16-byte unit u ^ (token / 2 % 4),
        eight dims a word, in order
  2048  K scales, four 16-bit words a token, one for each 32 dims
  2176  V scales, a 16-bit word a token

The eight codes of a word, from its lowest bits: dims 0, 2, 4, 6, 1, 3, 5, 7 of the eight.  A scale word is the bf16 pattern of s, whose last four bits (s has four significant bits) hold the zero
point z: element = s (code - z).
"""

import math
import random

import torch

own = False

D = 128      # head_dim
B = 16       # tokens of a block
RECORD = 2208
V_CODES, K_SCALES, V_SCALES = 1024, 2048, 2176
SCALE_LO, SCALE_HI = 2.0 ** -40, 2.0 ** 40


# ------------------------------------------------------------------------------ the cases --

def listed():
    return [
        # the new rows of a decode batch, one a sequence
        dict(name="store4_decode_256", kind="store", seqs=256, new=1, cached=2048, heads=12, kv=2, rot=128, layout="half"),
        # ragged prompts that continue cached tokens
        dict(name="store4_prefill_16384", kind="store", seqs=16, new=2048, cached=333, heads=32, kv=8, rot=128, layout="half"),
        # a cached prefix of one request brought back for another form of attention
        dict(name="read4_prefix_2000", kind="read", seqs=1, first=0, rows=2000, heads=12, kv=2),
        # the contexts of a batch of requests moved to a cache of another type
        dict(name="read4_mix64", kind="read", seqs=64, first=160, rows=2048, heads=32, kv=8),
        # the smallest serving call: one request, latency alone
        dict(name="decode4_b1_2048", kind="decode", seqs=1, ctx=2048, heads=12, kv=2, empty=False),
        # continuous batching: 64 requests with contexts of 64 to 4096 tokens
        dict(name="decode4_mix64", kind="decode", seqs=64, ctx=4096, heads=12, kv=2, empty=False),
        # few requests with long contexts
        dict(name="decode4_long4", kind="decode", seqs=4, ctx=32768, heads=32, kv=8, empty=False),
        # a small batch's fused step, part of the head rotated, adjacent pairs
        dict(name="step4_b8_1024", kind="step", seqs=8, ctx=1024, heads=28, kv=4, rot=64, layout="interleaved"),
        # continuous batching as the fused step of a wider model
        dict(name="step4_mix64", kind="step", seqs=64, ctx=4096, heads=32, kv=8, rot=128, layout="half"),
        # whole prompts
        dict(name="prefill4_4x2048", kind="prefill", seqs=4, new=2048, cached=0, heads=12, kv=2),
        # chunks that continue cached prompts
        dict(name="prefill4_16x256", kind="prefill", seqs=16, new=256, cached=1792, heads=12, kv=2),
        # a few proposed tokens of each request checked at once against a long context
        dict(name="prefill4_verify_8x5", kind="prefill", seqs=8, new=5, cached=6000, heads=28, kv=4),
    ]


HEADS = ((12, 2), (32, 8), (8, 8), (28, 4), (16, 2), (64, 8), (5, 1), (9, 3))


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("store", "store", "read", "decode", "decode", "step", "prefill", "prefill"))
    heads, kv = rng.choice(HEADS)
    form = dict(rot=16 * rng.randint(1, 8), layout=rng.choice(("half", "interleaved")))
    c = dict(kind=kind, heads=heads, kv=kv)
    if kind == "store":
        rows = max(1, 16384 * 40 // (heads + 2 * kv))
        seqs = _log(rng, 1, 512)
        new = _log(rng, 1, max(1, min(4096, rows // seqs, 32768 // seqs)))
        return dict(c, seqs=seqs, new=new, cached=_log(rng, 1, 4096) - 1, **form)
    if kind == "read":
        seqs = _log(rng, 1, 256)
        return dict(c, seqs=seqs, first=_log(rng, 1, 2048) - 1, rows=_log(rng, 1, min(16384, max(1, (1 << 19) // (seqs * kv)))))
    if kind in ("decode", "step"):
        seqs = _log(rng, 1, 256)
        ctx = _log(rng, 1, min(65536, max(1, (1 << 20) // (seqs * kv))))
        c = dict(c, seqs=seqs, ctx=ctx)
        return dict(c, empty=rng.random() < 0.3) if kind == "decode" else dict(c, **form)
    # prefill: bounded by the scores, seqs * heads * new * (cached + new)
    seqs = _log(rng, 1, 16)
    new = _log(rng, 1, 2048)
    while seqs * heads * new * new > 6e7:
        new = new * 2 // 3
    most = int(9e7 // (seqs * heads * new)) - new
    return dict(c, seqs=seqs, new=new, cached=_log(rng, 1, max(1, min(16384, most))) - 1)


TOKEN = RECORD / B           # bytes of a token and KV head in the cache, K and V


def work(case):
    """Bytes and operations of one pass: each input read once, each output written once."""
    c, k = case, case["kind"]
    if k == "store":
        rows = sum(_news(c))
        put = c["heads"] * D * 4 + c["kv"] * (D * 4 + TOKEN) + 4 * c["rot"] + 12
        return {"bytes": rows * (put + c["kv"] * D * 4), "flops": rows * (c["heads"] + c["kv"]) * c["rot"] * 3}
    if k == "read":
        rows = sum(_rows(c))
        return {"bytes": rows * c["kv"] * (TOKEN + 4 * D), "flops": rows * c["kv"] * 4 * D}
    if k in ("decode", "step"):
        tokens = sum(_contexts(c))
        extra = c["seqs"] * (c["kv"] * (8 * D + TOKEN) + 4 * c["rot"]) if k == "step" else 0
        return {"bytes": tokens * c["kv"] * TOKEN + tokens / 4 + 4 * c["seqs"] * c["heads"] * D + extra,
                "flops": 4.0 * tokens * c["heads"] * D}
    n, p = c["new"], c["cached"]
    pairs = c["seqs"] * (n * p + n * (n + 1) / 2)
    return {"bytes": c["seqs"] * ((n + p) * c["kv"] * TOKEN + 4 * n * c["heads"] * D), "flops": 4.0 * pairs * c["heads"] * D}


# ---------------------------------------------------------------------------- the inputs --

def _by_case(c):
    """The generator of a case's lengths: a case has the same lengths for every seed, in another order."""
    return random.Random(" ".join("%s=%s" % (k, c[k]) for k in sorted(c) if k != "name"))


def _contexts(c):
    """Context lengths of a decode batch: spread over ctx / 64 .. ctx, some empty where asked."""
    r = _by_case(c)
    lens = [r.randint(max(1, c["ctx"] // 64), c["ctx"]) if c["seqs"] > 1 else c["ctx"] for _ in range(c["seqs"])]
    return [0 if r.random() < 0.2 else n for n in lens] if c.get("empty") else lens


def _news(c):
    """New rows of each sequence of a store: 1, or half to all of `new`."""
    r = _by_case(c)
    return [r.randint((c["new"] + 1) // 2, c["new"]) for _ in range(c["seqs"])]


def _rows(c):
    """Rows of each sequence of a read: half to all of `rows`."""
    r = _by_case(c)
    return [r.randint((c["rows"] + 1) // 2, c["rows"]) if c["seqs"] > 1 else c["rows"] for _ in range(c["seqs"])]


def _shuffled(seed, *lists):
    """The requests of a batch in the seed's order."""
    order = list(range(len(lists[0])))
    random.Random(seed).shuffle(order)
    return [[a[i] for i in order] for a in lists]


def _cuda(a, dtype):
    return torch.tensor(a, dtype=dtype).cuda()


def _starts(lens):
    return torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32).cuda()


def _tables(gen, lens, num_blocks):
    """Block tables over a shuffled pool: each sequence's blocks in order, entries past them 0."""
    need = [(n + B - 1) // B for n in lens]
    perm = torch.randperm(num_blocks, generator=gen, device="cuda")[: sum(need)].to(torch.int32)
    at = torch.arange(max(max(need), 1), device="cuda")[None, :]
    table = torch.zeros((len(lens), at.shape[1]), dtype=torch.int32, device="cuda")
    table[at < _cuda(need, torch.int64)[:, None]] = perm
    return table


def _keys(gen, *shape):
    """Keys as models have them: a few channels far larger than the others."""
    x = torch.randn(shape + (D,), generator=gen, device="cuda")
    x[..., 5] *= 6.0
    x[..., 77] = x[..., 77] * 0.5 + 7.0
    return x.to(torch.bfloat16)


def _bf16(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)


def _cos_sin(positions, rot):
    w = 1e6 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * w[None, :]
    return torch.cat((a.cos(), a.sin()), dim=1).float().contiguous()


def _cache4(gen, num_blocks, kv):
    """A cache in use: every slot written."""
    cache = torch.zeros((num_blocks, kv, RECORD), dtype=torch.uint8, device="cuda")
    off = torch.arange(B, device="cuda")
    step = max(1, (1 << 25) // (kv * B * D))
    for b in range(0, num_blocks, step):
        n = min(step, num_blocks - b)
        blk = torch.arange(b, b + n, device="cuda").repeat_interleave(B)
        _put(cache, _keys(gen, n * B, kv), _bf16(gen, n * B, kv, D), blk, off.repeat(n))
    return cache


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = {"store": _prepare_store, "read": _prepare_read, "decode": _prepare_decode, "step": _prepare_decode,
          "prefill": _prepare_prefill}[case["kind"]](case, seed, gen)
    if own:                                    # what a serving loop keeps from step to step
        from paged_kv_cache_244_gb300 import binding
        st["pa"] = binding
        if case["kind"] in ("decode", "step"):
            st["ws"] = binding.decode_workspace_int4(st["q"], st["cache"], st["max_ctx"])
    return st


def _outputs(rows, kv):
    return dict(k_out=torch.empty((rows, kv, D), dtype=torch.bfloat16, device="cuda"),
                v_out=torch.empty((rows, kv, D), dtype=torch.bfloat16, device="cuda"))


def _prepare_store(c, seed, gen):
    r = _by_case(c)
    new, cached = _shuffled(seed, _news(c), [r.randint(0, c["cached"]) for _ in range(c["seqs"])])
    lens = [a + b for a, b in zip(cached, new)]
    num_blocks = sum((n + B - 1) // B for n in lens) + 5
    table = _tables(gen, lens, num_blocks)
    t, kv = sum(new), c["kv"]
    seq = torch.repeat_interleave(torch.arange(c["seqs"], device="cuda"), _cuda(new, torch.int64))
    start, first = _starts(new), _cuda(cached, torch.int32)
    pos = torch.arange(t, device="cuda") - start[seq] + first[seq]
    return dict(kind="store", layout=c["layout"], slots=table[seq, pos // B].to(torch.int64) * B + pos % B,
                pos=pos.to(torch.int32), q=_bf16(gen, t, c["heads"], D), k=_keys(gen, t, kv), v=_bf16(gen, t, kv, D),
                cos_sin=_cos_sin(max(lens), c["rot"]), q_out=torch.empty((t, c["heads"], D), dtype=torch.bfloat16, device="cuda"),
                cache=torch.zeros((num_blocks, kv, RECORD), dtype=torch.uint8, device="cuda"),
                table=table, start=start, first=first, max_rows=max(new), **_outputs(t, kv))


def _prepare_read(c, seed, gen):
    r = _by_case(c)
    rows, first = _shuffled(seed, _rows(c), [r.randint(c["first"] // 2, c["first"]) for _ in range(c["seqs"])])
    lens = [a + b for a, b in zip(first, rows)]
    num_blocks = sum((n + B - 1) // B for n in lens) + 3
    return dict(kind="read", cache=_cache4(gen, num_blocks, c["kv"]), table=_tables(gen, lens, num_blocks), start=_starts(rows),
                first=_cuda(first, torch.int32), max_rows=max(rows), **_outputs(sum(rows), c["kv"]))


def _prepare_decode(c, seed, gen):
    (lens,) = _shuffled(seed, _contexts(c))
    num_blocks = sum((n + B - 1) // B for n in lens) + 3
    st = dict(kind=c["kind"], q=_bf16(gen, c["seqs"], c["heads"], D), cache=_cache4(gen, num_blocks, c["kv"]),
              table=_tables(gen, lens, num_blocks), ctx=_cuda(lens, torch.int32), max_ctx=max(max(lens), 1), scale=D ** -0.5,
              out=torch.empty((c["seqs"], c["heads"], D), dtype=torch.bfloat16, device="cuda"))
    if c["kind"] == "step":
        st.update(k=_keys(gen, c["seqs"], c["kv"]), v=_bf16(gen, c["seqs"], c["kv"], D), cos_sin=_cos_sin(max(lens), c["rot"]),
                  layout=c["layout"], start=_starts([1] * c["seqs"]), first=st["ctx"] - 1, max_rows=1,
                  **_outputs(c["seqs"], c["kv"]))
    return st


def _prepare_prefill(c, seed, gen):
    r = _by_case(c)
    # chunks of one scheduler are alike; the last rows of a prompt and its cached part are ragged
    new = [c["new"] - (r.randint(0, c["new"] // 8) if s % 2 else 0) for s in range(c["seqs"])]
    new, cached = _shuffled(seed, new, [c["cached"] - (r.randint(0, c["cached"] // 8) if s % 2 else 0) for s in range(c["seqs"])])
    lens = [a + b for a, b in zip(cached, new)]
    num_blocks = sum((n + B - 1) // B for n in lens) + 3
    return dict(kind="prefill", q=_bf16(gen, sum(new), c["heads"], D), cache=_cache4(gen, num_blocks, c["kv"]),
                table=_tables(gen, lens, num_blocks), ctx=_cuda(lens, torch.int32), new=_cuda(new, torch.int64),
                start=_starts(new), max_new=max(new), max_ctx=max(lens), scale=D ** -0.5,
                out=torch.empty((sum(new), c["heads"], D), dtype=torch.bfloat16, device="cuda"))


# --------------------------------------------------------------------------- the operators --

def run(st):
    return (_run_own if own else _run_plain)[st["kind"]](st)


def _own_read(s):
    s["pa"].read_kv_int4(s["cache"], s["start"], s["first"], s["table"], s["max_rows"], k_out=s["k_out"], v_out=s["v_out"])
    return dict(k=s["k_out"], v=s["v_out"])


def _own_store(s):
    s["pa"].rope_kv_store_int4(s["q"], s["k"], s["v"], s["pos"], s["cos_sin"], s["slots"], s["cache"], layout=s["layout"],
                               q_out=s["q_out"])
    return dict(q=s["q_out"], **_own_read(s))


def _own_decode(s):
    return s["pa"].decode_int4(s["q"], s["cache"], s["table"], s["ctx"], s["max_ctx"], s["scale"], workspace=s["ws"], out=s["out"])


def _own_step(s):
    s["pa"].decode_step_int4(s["q"], s["k"], s["v"], s["cos_sin"], s["cache"], s["table"], s["ctx"], s["max_ctx"], s["scale"],
                             layout=s["layout"], workspace=s["ws"], out=s["out"])
    return dict(out=s["out"], **_own_read(s))


def _own_prefill(s):
    return s["pa"].prefill_int4(s["q"], s["start"], s["cache"], s["table"], s["ctx"], s["max_new"], s["max_ctx"], s["scale"],
                                out=s["out"])


def _quantised(x, groups):
    """bf16 rows [..., 128] as codes uint8 [..., 128] and scale words int16 [..., groups], one for each 128 / groups dims."""
    g = x.float().unflatten(-1, (groups, D // groups))
    real = torch.where(g.isfinite(), g, torch.zeros_like(g))
    lo, hi = real.amin(dim=-1).clamp(max=0.0), real.amax(dim=-1).clamp(min=0.0)
    m, e = torch.frexp((hi - lo).double() / 15.0)        # the smallest of four significant bits that is no less
    s = torch.ldexp(torch.ceil(m * 16.0), e - 4).clamp(SCALE_LO, SCALE_HI).float()
    z = torch.floor(-lo / s + 0.5).clamp(max=15.0)
    y = g / s[..., None]
    c = (torch.sign(y) * torch.floor(y.abs() + 0.5) + z[..., None]).nan_to_num(0.0).clamp(0.0, 15.0).to(torch.uint8)
    word = s.to(torch.bfloat16).view(torch.int16) | z.to(torch.int16)
    word = torch.where(g.isnan().any(dim=-1), torch.full_like(word, 0x7fc0), word)
    return c.flatten(-2), word


def _packed(codes):
    """Codes [..., 8 n] as the bytes [..., 4 n] of their words."""
    c = codes.unflatten(-1, (-1, 2, 2, 2)).movedim(-1, -3)     # dim 4 a + 2 b + o is nibble 4 o + 2 a + b
    return (c[..., 0] | (c[..., 1] << 4)).flatten(-3)


def _nibbles(b):
    """Bytes [..., 4 n] of words as codes [..., 8 n]."""
    c = torch.stack((b & 15, b >> 4), dim=-1).unflatten(-2, (-1, 2, 2))
    return c.movedim(-3, -1).flatten(-4)


def _put(cache, k, v, blk, off):
    """Rows k, v [T, kv, 128] quantised into slots `off` of blocks `blk` [T]."""
    t, kv, _ = k.shape
    kc, kw = _quantised(k, 4)
    vc, vw = _quantised(v, 1)
    kb = _packed(kc.unflatten(-1, (4, 4, 8)).transpose(-3, -2).flatten(-3))
    unit = torch.arange(4, device=k.device)[None, :] ^ (off[:, None] // 2 % 4)
    vb = _packed(vc).unflatten(-1, (4, 16)).gather(2, unit[:, None, :, None].expand(t, kv, 4, 16)).flatten(-2)
    b, h = blk[:, None, None], torch.arange(kv, device=k.device)[None, :, None]
    for part, at, x in ((0, 64, kb), (V_CODES, 64, vb), (K_SCALES, 8, kw.view(torch.uint8)), (V_SCALES, 2, vw.view(torch.uint8))):
        cache[b, h, (part + off[:, None] * at + torch.arange(at, device=k.device))[:, None, :]] = x


def _elements(cache, ids):
    """Elements (K, V) of blocks `ids` [S, n]: [S, kv, 16 n, 128] in fp32."""
    rec = cache[ids].transpose(1, 2)                      # [S, kv, n, record]
    shape = rec.shape[:3] + (B,)

    def words(part, groups):
        w = rec[..., part:part + 2 * B * groups].contiguous().view(torch.int16).view(shape + (groups, 1))
        return (w & ~15).view(torch.bfloat16).float(), (w & 15).float()

    s, z = words(K_SCALES, 4)
    k = _nibbles(rec[..., :V_CODES].reshape(shape + (4, 4, 4))).transpose(-3, -2).flatten(-2)    # [.., group, 32]
    k = ((k.float() - z) * s).flatten(-2)
    unit = torch.arange(4, device=rec.device)[None, :] ^ (torch.arange(B, device=rec.device)[:, None] // 2 % 4)
    v = _nibbles(rec[..., V_CODES:K_SCALES].reshape(shape + (4, 16)))
    v = v.gather(4, unit[:, :, None].expand(shape + (4, 32)))
    s, z = words(V_SCALES, 1)
    v = ((v.flatten(-2).float() - z[..., 0]) * s[..., 0])
    return k.flatten(2, 3), v.flatten(2, 3)


def _rotate(x, cos, sin, layout):
    """x [T, H, 128] bf16 rotated in 64 bits (a border of the bf16 rounding is not crossed), rounded to bf16."""
    half = cos.shape[1]
    y = x.double()
    c, n = cos.double()[:, None, :], sin.double()[:, None, :]
    if layout == "half":
        a, b = y[..., :half], y[..., half:2 * half]
        turned = torch.cat((a * c - b * n, b * c + a * n), dim=-1)
    else:
        a, b = y[..., 0:2 * half:2], y[..., 1:2 * half:2]
        turned = torch.stack((a * c - b * n, b * c + a * n), dim=-1).flatten(-2)
    return torch.cat((turned, y[..., 2 * half:]), dim=-1).to(torch.bfloat16)


def _store(s, pos, blk, off):
    """The rows into the cache; returns the rotated q."""
    half = s["cos_sin"].shape[1] // 2
    cs = s["cos_sin"][pos]
    cos, sin = cs[:, :half], cs[:, half:]
    _put(s["cache"], _rotate(s["k"], cos, sin, s["layout"]), s["v"], blk, off)
    return _rotate(s["q"], cos, sin, s["layout"])


def _plain_read(s):
    t = s["k_out"].shape[0]
    row = torch.arange(t, device=s["cache"].device)
    seq = torch.searchsorted(s["start"][1:].contiguous(), row.to(torch.int32), right=True)
    pos = row - s["start"][seq] + s["first"][seq]
    blk, off = s["table"][seq, pos // B].long(), pos % B
    h = torch.arange(s["cache"].shape[1], device=row.device)[None, :, None]

    def part(at, n):
        return s["cache"][blk[:, None, None], h, (at + off[:, None] * n + torch.arange(n, device=row.device))[:, None, :]]

    def values(codes, words):
        w = words.contiguous().view(torch.int16)
        c = codes.unflatten(-1, (w.shape[-1], -1)).float()
        return ((c - (w & 15).float()[..., None]) * (w & ~15).view(torch.bfloat16).float()[..., None]).flatten(-2)

    k = _nibbles(part(0, 64)).unflatten(-1, (4, 4, 8)).transpose(-3, -2).flatten(-3)
    unit = torch.arange(4, device=row.device)[None, :] ^ (off[:, None] // 2 % 4)
    v = part(V_CODES, 64).unflatten(-1, (4, 16))
    v = _nibbles(v.gather(2, unit[:, None, :, None].expand(v.shape)).flatten(-2))
    s["k_out"].copy_(values(k, part(K_SCALES, 8)))
    s["v_out"].copy_(values(v, part(V_SCALES, 2)))
    return dict(k=s["k_out"], v=s["v_out"])


def _plain_store(s):
    s["q_out"].copy_(_store(s, s["pos"].long(), s["slots"] // B, s["slots"] % B))
    return dict(q=s["q_out"], **_plain_read(s))


def _attend(q, k, v, live, scale):
    """softmax(scale q k^T) v over the live keys: q [S, kv, R, 128], live [S, 1 or kv, R, n]; rows with none give 0."""
    x = (q @ k.transpose(-1, -2)) * scale
    x = torch.where(live, x, torch.full_like(x, -torch.inf))
    top = x.amax(dim=-1, keepdim=True).clamp(min=torch.finfo(x.dtype).min)
    p = torch.exp(x - top)
    return (p @ v) / p.sum(dim=-1, keepdim=True).clamp(min=torch.finfo(x.dtype).tiny)


def _plain_decode(s, q=None):
    q = s["q"] if q is None else q
    n = (s["max_ctx"] + B - 1) // B
    k, v = _elements(s["cache"], s["table"][:, :n].long())
    live = (torch.arange(n * B, device=q.device)[None, :] < s["ctx"][:, None])[:, None, None, :]
    s["out"].copy_(_attend(q.float().view(q.shape[0], k.shape[1], -1, D), k, v, live, s["scale"]).view(q.shape))
    return s["out"]


def _plain_step(s):
    pos = s["ctx"].long() - 1
    blk = s["table"][torch.arange(pos.numel(), device=pos.device), pos // B].long()
    out = _plain_decode(s, _store(s, pos, blk, pos % B))
    return dict(out=out, **_plain_read(s))


def _plain_prefill(s):
    q, new, ctx = s["q"], s["new"], s["ctx"].long()
    n = (s["max_ctx"] + B - 1) // B
    k, v = _elements(s["cache"], s["table"][:, :n].long())
    seqs, kv = k.shape[:2]
    group = q.shape[1] // kv
    i = torch.arange(s["max_new"], device=q.device)
    real = i[None, :] < new[:, None]
    row = (s["start"][:-1].long()[:, None] + i[None, :]).clamp(max=q.shape[0] - 1)
    qq = q[row].float().view(seqs, s["max_new"], kv, group, D).permute(0, 2, 3, 1, 4).reshape(seqs, kv, -1, D)
    last = (ctx - new)[:, None] + i[None, :]
    live = torch.arange(n * B, device=q.device)[None, None, :] <= torch.where(real, last, torch.full_like(last, -1))[:, :, None]
    live = live[:, None, None].expand(seqs, 1, group, -1, -1).reshape(seqs, 1, group * s["max_new"], -1)
    o = _attend(qq, k, v, live, s["scale"]).view(seqs, kv, group, s["max_new"], D).permute(0, 3, 1, 2, 4)
    at = real.nonzero()
    s["out"][row[at[:, 0], at[:, 1]]] = o[at[:, 0], at[:, 1]].reshape(-1, kv * group, D).to(torch.bfloat16)
    return s["out"]


_run_own = {"store": _own_store, "read": _own_read, "decode": _own_decode, "step": _own_step, "prefill": _own_prefill}
_run_plain = {"store": _plain_store, "read": _plain_read, "decode": _plain_decode, "step": _plain_step, "prefill": _plain_prefill}


# ------------------------------------------------------------------ from the definitions --

def _exact_turn(x, cs, layout):
    """Each pair of each vector as a complex number times e^{i angle}, in 64 bits."""
    half = cs.shape[1] // 2
    turn = torch.complex(cs[:, :half].double(), cs[:, half:].double())[:, None, :]
    y = x.double().clone()
    one, two = (slice(0, half), slice(half, 2 * half)) if layout == "half" else (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
    z = torch.complex(y[..., one], y[..., two]) * turn
    y[..., one], y[..., two] = z.real, z.imag
    return y


#: The scales there are: m 2^e with m of four significant bits.
_SCALES = torch.tensor([m * 2.0 ** (e - 3) for e in range(-40, 40) for m in range(8, 16)] + [SCALE_HI], dtype=torch.float64)


def _exact_row(x, groups):
    """What rows x [..., 128] (finite) are as the cache holds them, in 64 bits."""
    g = x.double().unflatten(-1, (groups, D // groups))
    lo, hi = g.amin(dim=-1, keepdim=True).clamp(max=0), g.amax(dim=-1, keepdim=True).clamp(min=0)
    table = _SCALES.to(x.device)
    s = table[torch.searchsorted(15 * table, (hi - lo).float().double()).clamp(max=len(table) - 1)]
    z = ((-2 * lo / s + 1) / 2).floor().clamp(0, 15)
    y = g / s
    c = (torch.where(y < 0, (y - 0.5).ceil(), (y + 0.5).floor()) + z).clamp(0, 15)
    return ((c - z) * s).flatten(-2)


def _exact_blocks(cache, ids):
    """[kv, 16 n, 128] elements (K, V) of one sequence's blocks in 64 bits: bit fields of 32-bit words."""
    rec = cache[ids].contiguous()                         # [n, kv, record]
    w = rec.view(torch.int32).long() & 0xffffffff
    half = rec.view(torch.int16).long() & 0xffff
    dims = torch.arange(D, device=rec.device)
    tok = torch.arange(B, device=rec.device)[:, None]
    k_word = tok * 16 + 4 * (dims % 32 // 8) + dims // 32
    v_word = V_CODES // 4 + tok * 16 + 4 * ((dims // 32) ^ (tok // 2 % 4)) + dims % 32 // 8
    out = []
    for word, scale in ((k_word, K_SCALES // 2 + 4 * tok + dims // 32), (v_word, V_SCALES // 2 + tok + 0 * dims)):
        code = (w[:, :, word] >> (4 * (dims % 8 // 2 + 4 * (dims % 2)))) & 15
        m = half[:, :, scale]
        s = torch.ldexp(1.0 + (m >> 4 & 7).double() / 8, (m >> 7 & 255) - 127)
        out.append(((code - (m & 15)) * s).permute(1, 0, 2, 3).reshape(rec.shape[1], -1, D))
    return out


def _exact_rows(q, k, v, count, scale):
    """Attention of q [kv, R, 128] where row r of R sees the first count[r] keys, in 64 bits."""
    x = torch.einsum("grd,gtd->grt", q, k) * scale
    x = x.masked_fill(torch.arange(k.shape[1], device=q.device)[None, None, :] >= count[None, :, None], -math.inf)
    return torch.einsum("grt,gtd->grd", torch.softmax(x, dim=-1), v)


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "store":
        cs = s["cos_sin"][s["pos"].long()]
        # what is quantised is the rotated row as bf16
        k = _exact_row(_exact_turn(s["k"], cs, s["layout"]).to(torch.bfloat16), 4)
        return dict(q=_exact_turn(s["q"], cs, s["layout"]), k=k, v=_exact_row(s["v"], 1))
    tables = s["table"].long()
    if kind == "read":
        k, v = torch.empty(s["k_out"].shape, dtype=torch.float64, device="cuda"), torch.empty(s["k_out"].shape, dtype=torch.float64, device="cuda")
        start, first = s["start"].tolist(), s["first"].tolist()
        for i, f in enumerate(first):
            n = start[i + 1] - start[i]
            a, b = _exact_blocks(s["cache"], tables[i, : (f + n + B - 1) // B])
            k[start[i]:start[i + 1]], v[start[i]:start[i + 1]] = a[:, f:f + n].transpose(0, 1), b[:, f:f + n].transpose(0, 1)
        return dict(k=k, v=v)
    lens, kv = s["ctx"].tolist(), s["cache"].shape[1]
    q = s["q"].double()
    if kind == "step":
        # attention is with the rotated q as bf16, over the new token as the cache holds it
        cs = s["cos_sin"][s["ctx"].long() - 1]
        q = _exact_turn(s["q"], cs, s["layout"]).to(torch.bfloat16).double()
        k_new = _exact_row(_exact_turn(s["k"], cs, s["layout"]).to(torch.bfloat16), 4)
        v_new = _exact_row(s["v"], 1)
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    starts = s["start"].tolist() if kind == "prefill" else list(range(len(lens) + 1))
    for i, n in enumerate(lens):
        a, b = starts[i], starts[i + 1]
        if n == 0 or a == b:
            continue
        k, v = (x[:, :n] for x in _exact_blocks(s["cache"], tables[i, : (n + B - 1) // B]))
        if kind == "step":
            k[:, n - 1], v[:, n - 1] = k_new[i], v_new[i]
        rows = q[a:b].reshape(b - a, kv, -1, D).permute(1, 0, 2, 3)
        group = rows.shape[2]
        seen = torch.arange(n - (b - a) + 1, n + 1, device="cuda").repeat_interleave(group)
        o = _exact_rows(rows.reshape(kv, -1, D), k, v, seen, s["scale"])
        out[a:b] = o.reshape(kv, b - a, group, D).permute(1, 0, 2, 3).reshape(b - a, -1, D)
    return dict(out=out, k=k_new, v=v_new) if kind == "step" else out
