"""Operators of a serving step around a paged KV cache, in plain torch and as this framework's calls.

Three operators, each with the forms a serving loop needs:

  plan    the metadata of one step, built on the GPU from request lengths: blocks taken from a
          free list into the block tables, context lengths, row starts, positions and slots
  rotary  RoPE tables with long-context scaling, and the fused RoPE + cache store over the half
          and the interleaved layout and over part of the head
  block8  a KV cache of E4M3 codes with one power-of-two scale for each (block, KV head): the
          RoPE + quantising store, single-token decode, the fused decode step, and chunked prefill

Common shapes: head_dim 128, 16-token blocks, caches [num_blocks][kv_heads][16][128], scales
[num_blocks][kv_heads][2] (K, V), block tables [sequences][max_blocks] int32.
"""

import math
import random

import torch

own = False

D = 128      # head_dim
B = 16       # tokens of a block
E4M3_MAX = 448.0
SCALE_LO, SCALE_HI = 2.0 ** -40, 2.0 ** 40


# ------------------------------------------------------------------------------ the cases --

def listed():
    return [
        # one decode step's metadata of a busy server: every request gets one new token
        dict(name="plan_decode_256", kind="plan", seqs=256, cached=4096, new=1, heads=12, kv=2, short=0),
        # a prefill burst: many new prompts, some continuing a cached prefix, half a million rows
        dict(name="plan_prefill_512", kind="plan", seqs=512, cached=512, new=2048, heads=12, kv=2, short=0),
        # the table of a model stretched to 131,072 positions
        dict(name="table_yarn_131072", kind="table", positions=131072, rot=128, scaling="yarn", factor=32.0),
        # a decode batch of a model that rotates half of each head, adjacent pairs
        dict(name="store_interleaved_64", kind="rope", seqs=64, new=1, cached=4096, heads=32, kv=8, rot=64,
             layout="interleaved"),
        # a prefill of 32,768 rows with three quarters of the head rotated
        dict(name="store_half96_32768", kind="rope", seqs=16, new=2048, cached=0, heads=32, kv=8, rot=96, layout="half"),
        # the quantising store of a decode batch: one row into each sequence's newest block
        dict(name="store8_decode_256", kind="store8", seqs=256, new=1, cached=2048, heads=12, kv=2, rot=128, layout="half"),
        # the quantising store of a prefill of ragged prompts that continue cached tokens
        dict(name="store8_prefill_16384", kind="store8", seqs=16, new=1024, cached=333, heads=32, kv=8, rot=128,
             layout="half"),
        # the smallest serving call: one request, latency alone
        dict(name="decode8_b1_2048", kind="decode8", seqs=1, ctx=2048, heads=12, kv=2, empty=False),
        # continuous batching: 64 requests with contexts of 64 to 4096 tokens
        dict(name="decode8_mix64", kind="decode8", seqs=64, ctx=4096, heads=12, kv=2, empty=False),
        # the same step fused: rotate, quantise and store the new token, then attend
        dict(name="step8_mix64", kind="step8", seqs=64, ctx=4096, heads=32, kv=8, rot=128, layout="half"),
        # whole prompts
        dict(name="prefill8_4x2048", kind="prefill8", seqs=4, new=2048, cached=0, heads=12, kv=2),
        # chunks that continue cached prompts
        dict(name="prefill8_16x256", kind="prefill8", seqs=16, new=256, cached=1792, heads=12, kv=2),
    ]


HEADS = ((12, 2), (32, 8), (8, 8), (28, 4), (16, 2), (64, 8), (5, 1), (9, 3))


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("plan", "table", "rope", "store8", "decode8", "decode8", "step8", "prefill8", "prefill8"))
    heads, kv = rng.choice(HEADS)
    rot = 16 * rng.randint(1, 8)
    layout = rng.choice(("half", "interleaved"))
    if kind == "plan":
        seqs = _log(rng, 1, 4096)
        new = _log(rng, 1, max(1, min(4096, 800000 // seqs)))
        return dict(kind=kind, seqs=seqs, cached=_log(rng, 1, 8192), new=new, heads=heads, kv=kv, short=rng.choice((0, 0, 1)))
    if kind == "table":
        return dict(kind=kind, positions=_log(rng, 100, 131072), rot=rot, scaling=rng.choice(("none", "linear", "ntk", "yarn", "banded")),
                    factor=round(rng.uniform(1.5, 40.0), 3))
    if kind in ("rope", "store8"):
        rows = max(1, 32768 * 40 // (heads + 2 * kv))
        seqs = _log(rng, 1, 512)
        new = _log(rng, 1, max(1, min(4096, rows // seqs, 32768 // seqs)))
        return dict(kind=kind, seqs=seqs, new=new, cached=_log(rng, 1, 4096) - 1, heads=heads, kv=kv, rot=rot, layout=layout)
    if kind in ("decode8", "step8"):
        seqs = _log(rng, 1, 256)
        ctx = _log(rng, 1, min(65536, max(1, (1 << 20) // (seqs * kv))))
        c = dict(kind=kind, seqs=seqs, ctx=ctx, heads=heads, kv=kv)
        return dict(c, empty=rng.random() < 0.3) if kind == "decode8" else dict(c, rot=rot, layout=layout)
    # prefill: bounded by the scores, seqs * heads * new * (cached + new)
    seqs = _log(rng, 1, 16)
    new = _log(rng, 1, 2048)
    while seqs * heads * new * new > 6e7:
        new = new * 2 // 3
    most = int(9e7 // (seqs * heads * new)) - new
    cached = _log(rng, 1, max(1, min(16384, most))) - 1
    return dict(kind=kind, seqs=seqs, new=new, cached=cached, heads=heads, kv=kv)


def work(case):
    """Bytes and operations of one pass: each input read once, each output written once."""
    c, k = case, case["kind"]
    if k == "plan":
        rows = c["seqs"] * (c["new"] + 1) / 2
        blocks = rows / B
        # lengths in, lengths and starts out, positions and slots out, the blocks' ids in and out
        return {"bytes": 20 * c["seqs"] + 12 * rows + 8 * blocks, "flops": 4 * rows}
    if k == "table":
        n = c["positions"] * c["rot"]
        return {"bytes": 4 * n, "flops": 20 * n}
    if k in ("rope", "store8"):
        rows = c["seqs"] * (c["new"] + 1) / 2 if c["new"] > 1 else c["seqs"]
        per = c["heads"] * D * 4 + 2 * c["kv"] * D * (4 if k == "rope" else 3) + 4 * c["rot"] + 12
        return {"bytes": rows * per, "flops": rows * (c["heads"] + c["kv"]) * c["rot"] * 3}
    if k in ("decode8", "step8"):
        tokens = sum(_contexts(c))
        rw = 2 * c["seqs"] * c["heads"] * D * 2
        extra = c["seqs"] * (2 * c["kv"] * D * 3 + 4 * c["rot"]) if k == "step8" else 0
        return {"bytes": tokens * c["kv"] * 2 * (D + 0.5 / 2) + tokens / 4 + rw + extra, "flops": 4.0 * tokens * c["heads"] * D}
    n, p = c["new"], c["cached"]
    pairs = c["seqs"] * (n * p + n * (n + 1) / 2)
    kvb = c["seqs"] * (n + p) * c["kv"] * 2 * (D + 0.25)
    return {"bytes": kvb + 2 * c["seqs"] * n * c["heads"] * D * 2, "flops": 4.0 * pairs * c["heads"] * D}


# ---------------------------------------------------------------------------- the inputs --

def _by_case(c):
    """The generator of a case's lengths: a case has the same lengths for every seed, in another order."""
    return random.Random(" ".join("%s=%s" % (k, c[k]) for k in sorted(c) if k != "name"))


def _contexts(c):
    """Context lengths of a decode batch: spread over ctx / 64 .. ctx, some empty where asked."""
    r = _by_case(c)
    lens = [r.randint(max(1, c["ctx"] // 64), c["ctx"]) if c["seqs"] > 1 else c["ctx"] for _ in range(c["seqs"])]
    if c.get("empty"):
        lens = [0 if r.random() < 0.2 else n for n in lens]
    return lens


def _shuffled(seed, *lists):
    """The requests of a batch in the seed's order."""
    order = list(range(len(lists[0])))
    random.Random(seed).shuffle(order)
    return [[a[i] for i in order] for a in lists]


def _cuda(a, dtype):
    return torch.tensor(a, dtype=dtype).cuda()


def _tables(gen, lens, num_blocks):
    """Block tables over a shuffled pool: each sequence's blocks in order, entries past them 0."""
    need = [(n + B - 1) // B for n in lens]
    width = max(max(need), 1)
    perm = torch.randperm(num_blocks, generator=gen, device="cuda")[: sum(need)].to(torch.int32)
    at = torch.arange(width, device="cuda")[None, :]
    cnt = _cuda(need, torch.int64)[:, None]
    table = torch.zeros((len(lens), width), dtype=torch.int32, device="cuda")
    table[at < cnt] = perm
    return table


def _pow2_scale(amax):
    """The smallest power of two s with amax <= 448 s, within [2^-40, 2^40] (fp32 in, fp32 out)."""
    m, e = torch.frexp(amax)            # amax = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    s = torch.ldexp(torch.ones_like(amax), e - 9 + (m > 0.875).to(e.dtype))
    return torch.where(amax > 0, s, torch.zeros_like(s)).clamp(SCALE_LO, SCALE_HI)


def _codes(x, inv):
    """E4M3 codes (as torch's type) of x * inv, saturating."""
    return (x * inv).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _cache8(gen, num_blocks, kv):
    """A cache of E4M3 codes whose blocks differ in magnitude, with the scales they stand at."""
    codes, scales = [], []
    for _ in range(2):
        spread = torch.exp(0.7 * torch.randn((num_blocks, kv, 1, 1), generator=gen, device="cuda"))
        x = torch.randn((num_blocks, kv, B, D), generator=gen, device="cuda") * spread
        s = _pow2_scale(x.abs().amax(dim=(2, 3)))
        codes.append(_codes(x, 1.0 / s[:, :, None, None]).view(torch.uint8))
        scales.append(s)
    return codes[0], codes[1], torch.stack(scales, dim=2).contiguous()


def _cos_sin(positions, rot):
    w = 1e6 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * w[None, :]
    return torch.cat((a.cos(), a.sin()), dim=1).float().contiguous()


def _bf16(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = {"plan": _prepare_plan, "table": _prepare_table, "rope": _prepare_store, "store8": _prepare_store,
          "decode8": _prepare_decode, "step8": _prepare_decode, "prefill8": _prepare_prefill}[case["kind"]](case, seed, gen)
    if own:                                    # what a serving loop keeps from step to step
        from paged_kv_cache_244_gb300 import binding
        st["pa"] = binding
        if case["kind"] == "plan":
            st["out"] = binding.step_plan(case["seqs"], st["rows"])
        if case["kind"] in ("decode8", "step8"):
            st["ws"] = binding.decode_workspace(st["q"], st["k_cache"], st["max_ctx"])
    return st


def _prepare_plan(c, seed, gen):
    r = _by_case(c)
    cached = [r.randint(0, c["cached"]) if c["new"] > 1 else r.randint(c["cached"] // 64, c["cached"]) for _ in range(c["seqs"])]
    cached, new = _shuffled(seed, cached, [r.randint(1, c["new"]) for _ in range(c["seqs"])])
    have = sum((n + B - 1) // B for n in cached)
    need = sum((n + m + B - 1) // B for n, m in zip(cached, new)) - have
    # a pool with room, or (short) one whose free list ends in the middle of the batch
    free = max(1, need * 2 // 3) if c["short"] else need + 1000
    num_blocks = have + free
    perm = torch.randperm(num_blocks, generator=gen, device="cuda").to(torch.int32)
    width = max((n + m + B - 1) // B for n, m in zip(cached, new))
    table = torch.full((c["seqs"], width), -1, dtype=torch.int32, device="cuda")
    at = torch.arange(width, device="cuda")[None, :]
    cnt = _cuda([(n + B - 1) // B for n in cached], torch.int64)[:, None]
    table[at < cnt] = perm[:have]
    rows = sum(new) + 7                                  # a captured step is padded to a fixed number of rows
    i32 = dict(dtype=torch.int32, device="cuda")
    return dict(kind="plan", cached=_cuda(cached, torch.int32), new=_cuda(new, torch.int32), table=table, rows=rows,
                free=perm[have:].contiguous(), num_free=torch.full((1,), free, **i32), num_blocks=num_blocks,
                num_free_out=torch.empty((1,), **i32))


def _prepare_table(c, seed, gen):
    r = random.Random(seed)
    theta = r.uniform(9e3, 1.1e6)
    return dict(kind="table", positions=c["positions"], rot=c["rot"], scaling=c["scaling"], factor=c["factor"], theta=theta,
                original=4096, low=1.0, high=32.0 if c["scaling"] == "yarn" else 4.0,
                out=torch.empty((c["positions"], c["rot"]), dtype=torch.float32, device="cuda"))


def _prepare_store(c, seed, gen):
    r = _by_case(c)
    new = [r.randint(1, c["new"]) for _ in range(c["seqs"])]
    new, cached = _shuffled(seed, new, [r.randint(0, c["cached"]) for _ in range(c["seqs"])])
    lens = [a + b for a, b in zip(cached, new)]
    num_blocks = sum((n + B - 1) // B for n in lens) + 5
    table = _tables(gen, lens, num_blocks)
    t = sum(new)
    seq = torch.repeat_interleave(torch.arange(c["seqs"], device="cuda"), _cuda(new, torch.int64))
    first = torch.tensor([0] + new[:-1]).cumsum(0).cuda()
    pos = torch.arange(t, device="cuda") - first[seq] + _cuda(cached, torch.int64)[seq]
    slots = table[seq, pos // B].to(torch.int64) * B + pos % B
    slots[torch.rand(t, generator=gen, device="cuda") < 0.01] = -1      # some rows are padding
    kv, bf = c["kv"], torch.bfloat16
    st = dict(kind=c["kind"], layout=c["layout"], slots=slots, pos=pos.to(torch.int32),
              q=_bf16(gen, t, c["heads"], D), k=_bf16(gen, t, kv, D), v=_bf16(gen, t, kv, D),
              cos_sin=_cos_sin(max(lens), c["rot"]), q_out=torch.empty((t, c["heads"], D), dtype=bf, device="cuda"))
    if c["kind"] == "rope":
        st.update(k_cache=torch.zeros((num_blocks, kv, B, D), dtype=bf, device="cuda"),
                  v_cache=torch.zeros((num_blocks, kv, B, D), dtype=bf, device="cuda"))
    else:
        kc, vc, sc = _cache8(gen, num_blocks, kv)
        st.update(k_cache=kc, v_cache=vc, kv_scale=sc)
    return st


def _prepare_decode(c, seed, gen):
    (lens,) = _shuffled(seed, _contexts(c))
    num_blocks = sum((n + B - 1) // B for n in lens) + 3
    kc, vc, sc = _cache8(gen, num_blocks, c["kv"])
    st = dict(kind=c["kind"], q=_bf16(gen, c["seqs"], c["heads"], D), k_cache=kc, v_cache=vc, kv_scale=sc,
              table=_tables(gen, lens, num_blocks), ctx=_cuda(lens, torch.int32), max_ctx=max(max(lens), 1), scale=D ** -0.5,
              out=torch.empty((c["seqs"], c["heads"], D), dtype=torch.bfloat16, device="cuda"))
    if c["kind"] == "step8":
        st.update(k=_bf16(gen, c["seqs"], c["kv"], D), v=_bf16(gen, c["seqs"], c["kv"], D),
                  cos_sin=_cos_sin(max(lens), c["rot"]), layout=c["layout"])
    return st


def _prepare_prefill(c, seed, gen):
    r = _by_case(c)
    # chunks of one scheduler are alike; the last rows of a prompt and its cached part are ragged
    new = [c["new"] - (r.randint(0, c["new"] // 8) if s % 2 else 0) for s in range(c["seqs"])]
    new, cached = _shuffled(seed, new, [c["cached"] - (r.randint(0, c["cached"] // 8) if s % 2 else 0) for s in range(c["seqs"])])
    lens = [a + b for a, b in zip(cached, new)]
    num_blocks = sum((n + B - 1) // B for n in lens) + 3
    kc, vc, sc = _cache8(gen, num_blocks, c["kv"])
    return dict(kind="prefill8", q=_bf16(gen, sum(new), c["heads"], D), k_cache=kc, v_cache=vc, kv_scale=sc,
                table=_tables(gen, lens, num_blocks), ctx=_cuda(lens, torch.int32), new=_cuda(new, torch.int64),
                q_start=torch.tensor([0] + new).cumsum(0).to(torch.int32).cuda(), max_new=max(new), max_ctx=max(lens),
                scale=D ** -0.5, out=torch.empty((sum(new), c["heads"], D), dtype=torch.bfloat16, device="cuda"))


# --------------------------------------------------------------------------- the operators --

def run(st):
    return (_run_own if own else _run_plain)[st["kind"]](st)


def _own_plan(s):
    p = s["pa"].plan_step(s["cached"], s["new"], s["table"], s["free"], s["num_free"], s["num_blocks"], s["rows"],
                          num_free_out=s["num_free_out"], plan=s["out"])
    return dict(context_lens=p.context_lens, q_start=p.q_start, positions=p.positions, slots=p.slot_mapping,
                granted=p.granted, table=s["table"], num_free=s["num_free_out"])


def _own_table(s):
    return s["pa"].rope_table(s["positions"], s["rot"], s["theta"], scaling=s["scaling"], factor=s["factor"],
                              original_max_pos=s["original"], low=s["low"], high=s["high"], out=s["out"])


def _own_rope(s):
    s["pa"].rope_kv_store_form(s["q"], s["k"], s["v"], s["pos"], s["cos_sin"], s["slots"], s["k_cache"], s["v_cache"],
                               layout=s["layout"], q_out=s["q_out"])
    return dict(q=s["q_out"], k_cache=s["k_cache"], v_cache=s["v_cache"])


def _own_store8(s):
    s["pa"].rope_kv_store_fp8_block(s["q"], s["k"], s["v"], s["pos"], s["cos_sin"], s["slots"], s["k_cache"], s["v_cache"],
                                    s["kv_scale"], layout=s["layout"], q_out=s["q_out"])
    return dict(q=s["q_out"], **_values(s))


def _own_decode(s):
    return s["pa"].decode_fp8_block(s["q"], s["k_cache"], s["v_cache"], s["kv_scale"], s["table"], s["ctx"], s["max_ctx"],
                                    s["scale"], workspace=s["ws"], out=s["out"])


def _own_step(s):
    out = s["pa"].decode_step_fp8_block(s["q"], s["k"], s["v"], s["cos_sin"], s["k_cache"], s["v_cache"], s["kv_scale"],
                                        s["table"], s["ctx"], s["max_ctx"], s["scale"], layout=s["layout"],
                                        workspace=s["ws"], out=s["out"])
    return dict(out=out, **_values(s))


def _own_prefill(s):
    return s["pa"].prefill_fp8_block(s["q"], s["q_start"], s["k_cache"], s["v_cache"], s["kv_scale"], s["table"], s["ctx"],
                                     s["max_new"], s["max_ctx"], s["scale"], out=s["out"])


def _values(s):
    """The caches a call has written: each code as the E4M3 value it is (times its block's scale: the element)."""
    f8 = torch.float8_e4m3fn
    return dict(k_codes=s["k_cache"].view(f8), v_codes=s["v_cache"].view(f8), kv_scale=s["kv_scale"])


def _plain_plan(s):
    cached, new, table = s["cached"].long(), s["new"].long(), s["table"]
    width, t = table.shape[1], s["rows"]
    rows = torch.where((new >= 0) & (new <= t), new, torch.zeros_like(new))
    end = rows.cumsum(0)
    good = (cached >= 0) & (new >= 0) & (new <= t) & (cached + new <= width * B) & (end <= t)
    old = (cached + B - 1) // B
    need = torch.where(good, (cached + new + B - 1) // B - old, torch.zeros_like(new))
    upto = need.cumsum(0)
    avail = s["num_free"].long()
    granted = good & ((need == 0) | (upto <= avail))
    ctx = torch.where(granted, cached + new, torch.zeros_like(new))
    at = torch.arange(width, device=table.device)[None, :]
    fresh = granted[:, None] & (at >= old[:, None]) & (at < (old + need)[:, None])
    idx = avail - 1 - ((upto - need)[:, None] + at - old[:, None])
    table.copy_(torch.where(fresh, s["free"][idx.clamp(0, s["free"].numel() - 1)], table))
    row = torch.arange(t, device=table.device)
    seq = torch.searchsorted(end, row, right=True)
    live = seq < end.numel()
    seq = seq.clamp(max=end.numel() - 1)
    live = live & granted[seq]
    pos = torch.where(live, row - (end - rows)[seq] + cached[seq], torch.zeros_like(row))
    slot = torch.where(live, table[seq, pos // B].long() * B + pos % B, torch.full_like(row, -1))
    start = torch.cat((torch.zeros_like(end[:1]), end))
    taken = torch.where(granted, need, torch.zeros_like(need)).sum()
    i32 = torch.int32
    return dict(context_lens=ctx.to(i32), q_start=start.to(i32), positions=pos.to(i32), slots=slot, granted=granted.to(i32),
                table=table, num_free=(avail - taken).to(i32))


def _frequencies(s):
    """The angles per position of each pair, in 64 bits, and the factor on cos and sin."""
    rot, theta, f, old = s["rot"], s["theta"], s["factor"], s["original"]
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    w = torch.exp(-2.0 * i / rot * math.log(theta))
    if s["scaling"] == "linear":
        return w / f, 1.0
    if s["scaling"] == "ntk":
        return torch.exp(-2.0 * i / rot * math.log(theta * f ** (rot / (rot - 2.0)))), 1.0
    if s["scaling"] == "yarn":
        at = [rot * math.log(old / (2.0 * math.pi * turns)) / (2.0 * math.log(theta)) for turns in (s["high"], s["low"])]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        ramp = ((i - lo) / (hi - lo if hi != lo else 0.001)).clamp(0.0, 1.0)
        return w / f * ramp + w * (1.0 - ramp), 0.1 * math.log(f) + 1.0
    if s["scaling"] == "banded":
        turns = old * w / (2.0 * math.pi)                # of one pair over the original context
        mix = ((turns - s["low"]) / (s["high"] - s["low"])).clamp(0.0, 1.0)
        return w / f * (1.0 - mix) + w * mix, 1.0
    return w, 1.0


def _plain_table(s):
    w, m = _frequencies(s)
    a = torch.arange(s["positions"], dtype=torch.float64, device="cuda")[:, None] * w[None, :]
    return (torch.cat((a.cos(), a.sin()), dim=1) * m).float()


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


def _plain_rope(s):
    half = s["cos_sin"].shape[1] // 2
    cs = s["cos_sin"][s["pos"].long()]
    cos, sin = cs[:, :half], cs[:, half:]
    s["q_out"].copy_(_rotate(s["q"], cos, sin, s["layout"]))
    k = _rotate(s["k"], cos, sin, s["layout"])
    keep = (s["slots"] >= 0).nonzero()[:, 0]
    blk, off = s["slots"][keep] // B, s["slots"][keep] % B
    s["k_cache"][blk, :, off] = k[keep]
    s["v_cache"][blk, :, off] = s["v"][keep]
    return dict(q=s["q_out"], k_cache=s["k_cache"], v_cache=s["v_cache"])


def _put8(cache, scale, x, blk, off):
    """Quantises rows x [T, kv, 128] into their blocks; a block's scale is set by its first slot's
    call, and otherwise grows when it has to, with the codes it holds coded anew."""
    ids, run = torch.unique_consecutive(blk, return_inverse=True)
    x = x.float()
    a = torch.where(x.isfinite(), x.abs(), torch.zeros_like(x)).amax(dim=2)
    top = torch.zeros((ids.numel(), x.shape[1]), device=x.device).scatter_reduce_(0, run[:, None].expand_as(a), a, "amax")
    want = _pow2_scale(top)
    begun = torch.zeros(ids.numel(), device=x.device).scatter_reduce_(0, run, (off == 0).float(), "amax") > 0
    old = scale[ids]
    now = torch.where(begun[:, None] | ~(old > want), want, old)
    held = cache[ids].view(torch.float8_e4m3fn).float()
    grown = (~begun[:, None] & (now > old))[:, :, None, None]
    cache[ids] = torch.where(grown, _codes(held, (old / now)[:, :, None, None]).view(torch.uint8), cache[ids])
    scale[ids] = now
    cache[blk, :, off] = _codes(x, (1.0 / now)[run][:, :, None]).view(torch.uint8)


def _store8(s, q, pos, blk, off, keep):
    half = s["cos_sin"].shape[1] // 2
    cs = s["cos_sin"][pos]
    cos, sin = cs[:, :half], cs[:, half:]
    k = _rotate(s["k"], cos, sin, s["layout"])
    _put8(s["k_cache"], s["kv_scale"][..., 0], k[keep], blk, off)
    _put8(s["v_cache"], s["kv_scale"][..., 1], s["v"][keep], blk, off)
    return _rotate(q, cos, sin, s["layout"])


def _plain_store8(s):
    keep = (s["slots"] >= 0).nonzero()[:, 0]
    slots = s["slots"][keep]
    s["q_out"].copy_(_store8(s, s["q"], s["pos"].long(), slots // B, slots % B, keep))
    return dict(q=s["q_out"], **_values(s))


def _gathered(cache, scale, ids):
    """The elements of the blocks `ids` [S, n]: [S, kv, 16 n, 128] in fp32."""
    x = cache[ids].view(torch.float8_e4m3fn).float() * scale[ids][..., None, None]
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)


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
    ids = s["table"][:, :n].long()
    k, v = _gathered(s["k_cache"], s["kv_scale"][..., 0], ids), _gathered(s["v_cache"], s["kv_scale"][..., 1], ids)
    kv = k.shape[1]
    live = (torch.arange(n * B, device=q.device)[None, :] < s["ctx"][:, None])[:, None, None, :]
    s["out"].copy_(_attend(q.float().view(q.shape[0], kv, -1, D), k, v, live, s["scale"]).view(q.shape))
    return s["out"]


def _plain_step(s):
    pos = s["ctx"].long() - 1
    rows = torch.arange(pos.numel(), device=pos.device)
    blk = s["table"][rows, pos // B].long()
    q = _store8(s, s["q"], pos, blk, pos % B, rows)
    return dict(out=_plain_decode(s, q), **_values(s))


def _plain_prefill(s):
    q, new, ctx = s["q"], s["new"], s["ctx"].long()
    n = (s["max_ctx"] + B - 1) // B
    ids = s["table"][:, :n].long()
    k, v = _gathered(s["k_cache"], s["kv_scale"][..., 0], ids), _gathered(s["v_cache"], s["kv_scale"][..., 1], ids)
    seqs, kv, group = ids.shape[0], k.shape[1], q.shape[1] // k.shape[1]
    i = torch.arange(s["max_new"], device=q.device)
    real = i[None, :] < new[:, None]
    row = (s["q_start"][:-1].long()[:, None] + i[None, :]).clamp(max=q.shape[0] - 1)
    qq = q[row].float().view(seqs, s["max_new"], kv, group, D).permute(0, 2, 3, 1, 4).reshape(seqs, kv, -1, D)
    last = (ctx - new)[:, None] + i[None, :]
    live = torch.arange(n * B, device=q.device)[None, None, :] <= torch.where(real, last, torch.full_like(last, -1))[:, :, None]
    live = live[:, None, None].expand(seqs, 1, group, -1, -1).reshape(seqs, 1, group * s["max_new"], -1)
    o = _attend(qq, k, v, live, s["scale"]).view(seqs, kv, group, s["max_new"], D).permute(0, 3, 1, 2, 4)
    at = real.nonzero()
    s["out"][row[at[:, 0], at[:, 1]]] = o[at[:, 0], at[:, 1]].reshape(-1, kv * group, D).to(torch.bfloat16)
    return s["out"]


_run_own = {"plan": _own_plan, "table": _own_table, "rope": _own_rope, "store8": _own_store8, "decode8": _own_decode,
            "step8": _own_step, "prefill8": _own_prefill}
_run_plain = {"plan": _plain_plan, "table": _plain_table, "rope": _plain_rope, "store8": _plain_store8,
              "decode8": _plain_decode, "step8": _plain_step, "prefill8": _plain_prefill}


# ------------------------------------------------------------------ from the definitions --

_E4M3 = [((c >> 3 & 15) and (1 + (c & 7) / 8) * 2.0 ** ((c >> 3 & 15) - 7) or (c & 7) / 8 * 2.0 ** -6) * (-1) ** (c >> 7)
         if c & 127 != 127 else math.nan for c in range(256)]


def _exact_turn(x, cs, layout):
    """Each pair of each vector as a complex number times e^{i angle}, in 64 bits."""
    half = cs.shape[1] // 2
    turn = torch.complex(cs[:, :half].double(), cs[:, half:].double())[:, None, :]
    y = x.double().clone()
    one, two = (slice(0, half), slice(half, 2 * half)) if layout == "half" else (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
    z = torch.complex(y[..., one], y[..., two]) * turn
    y[..., one], y[..., two] = z.real, z.imag
    return y


_E4M3_UP = torch.tensor(_E4M3[:127], dtype=torch.float64)                 # 0 .. 448


def _exact_code(x):
    """The nearest E4M3 code of each value (the even one of two as near), in 64 bits; beyond 448: 448."""
    up = _E4M3_UP.to(x.device)
    a = x.abs().clamp(max=E4M3_MAX)
    hi = torch.searchsorted(up, a).clamp(min=1)
    low, high = a - up[hi - 1], up[hi] - a
    code = torch.where((high < low) | ((high == low) & (hi % 2 == 0)), hi, hi - 1)
    return (code + 128 * (x < 0).long()).to(torch.uint8)


def _exact_append(codes, scale, x, off):
    """One block [kv, 16, 128] after row x [kv, 128] went to slot off: (codes, scales)."""
    value = torch.tensor(_E4M3, dtype=torch.float64, device=codes.device)
    out, now = codes.clone(), scale.double().clone()
    for h, a in enumerate(x.double().abs().amax(dim=1).tolist()):
        s = SCALE_LO
        while s < SCALE_HI and a > E4M3_MAX * s:
            s *= 2
        if off > 0 and now[h] >= s:
            s = float(now[h])
        elif off > 0:
            out[h] = _exact_code(value[codes[h].long()] * (float(now[h]) / s))
        now[h] = s
        out[h, off] = _exact_code(x[h].double() / s)
    return out, now.float()


def _exact_elements(codes, scale, ids):
    """[kv, 16 n, 128] elements of one sequence's blocks in 64 bits."""
    value = torch.tensor(_E4M3, dtype=torch.float64, device=codes.device)
    x = value[codes[ids].long()] * scale[ids].double()[:, :, None, None]
    return x.permute(1, 0, 2, 3).reshape(codes.shape[1], -1, D)


def _exact_rows(q, k, v, count, scale):
    """Attention of q [kv, R, 128] where row r of R sees the first count[r] keys, in 64 bits."""
    x = torch.einsum("grd,gtd->grt", q, k) * scale
    x = x.masked_fill(torch.arange(k.shape[1], device=q.device)[None, None, :] >= count[None, :, None], -math.inf)
    return torch.einsum("grt,gtd->grd", torch.softmax(x, dim=-1), v)


def exact(case, seed):
    kind = case["kind"]
    if kind == "plan":
        return None                                       # whole numbers
    s = prepare(case, seed)
    if kind == "table":
        w, m = _exact_frequencies(s)
        a = torch.arange(s["positions"], dtype=torch.float64)[:, None] * w[None, :]
        return (torch.cat((torch.cos(a), torch.sin(a)), dim=1) * m)
    if kind in ("rope", "store8"):
        cs = s["cos_sin"][s["pos"].long()]
        q = _exact_turn(s["q"], cs, s["layout"])
        if kind == "store8":
            return dict(q=q, k_codes=None, v_codes=None, kv_scale=None)      # codes and scales are roundings
        k, kc, vc = _exact_turn(s["k"], cs, s["layout"]), s["k_cache"].double(), s["v_cache"].double()
        for t, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                kc[slot // B, :, slot % B] = k[t]
                vc[slot // B, :, slot % B] = s["v"][t].double()
        return dict(q=q, k_cache=kc, v_cache=vc)
    kv, scale = s["k_cache"].shape[1], s["scale"]
    lens, tables = s["ctx"].tolist(), s["table"].long()
    if kind == "step8":
        # the operator attends with the rotated q as bf16, over the new token as the cache holds it
        cs = s["cos_sin"][s["ctx"].long() - 1]
        q = _exact_turn(s["q"], cs, s["layout"]).to(torch.bfloat16).double()
        k = _exact_turn(s["k"], cs, s["layout"]).to(torch.bfloat16)
        for i, n in enumerate(lens):
            at = int(tables[i, (n - 1) // B])
            for j, (name, x) in enumerate((("k_cache", k), ("v_cache", s["v"]))):
                s[name][at], s["kv_scale"][at, :, j] = _exact_append(s[name][at], s["kv_scale"][at, :, j], x[i], (n - 1) % B)
    else:
        q = s["q"].double()
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    starts = s["q_start"].tolist() if kind == "prefill8" else list(range(len(lens) + 1))
    for i, n in enumerate(lens):
        a, b = starts[i], starts[i + 1]
        if n == 0 or a == b:
            continue
        ids = tables[i, : (n + B - 1) // B]
        k, v = (_exact_elements(s[c], s["kv_scale"][..., j], ids)[:, :n] for j, c in enumerate(("k_cache", "v_cache")))
        rows = q[a:b].reshape(b - a, kv, -1, D).permute(1, 0, 2, 3)
        group = rows.shape[2]
        seen = torch.arange(n - (b - a) + 1, n + 1, device="cuda").repeat_interleave(group)
        o = _exact_rows(rows.reshape(kv, -1, D), k, v, seen, scale)
        out[a:b] = o.reshape(kv, b - a, group, D).permute(1, 0, 2, 3).reshape(b - a, -1, D)
    return dict(out=out, k_codes=None, v_codes=None, kv_scale=None) if kind == "step8" else out


def _exact_frequencies(s):
    """One pair at a time, as the scalings are defined."""
    rot, theta, f, old, kind = s["rot"], s["theta"], s["factor"], s["original"], s["scaling"]
    if kind == "ntk":
        theta *= f ** (rot / (rot - 2))
    w = [theta ** (-2 * i / rot) for i in range(rot // 2)]
    if kind == "linear":
        w = [x / f for x in w]
    if kind == "yarn":
        def place(turns):
            return rot * math.log(old / (turns * 2 * math.pi)) / (2 * math.log(theta))
        first, last = max(math.floor(place(s["high"])), 0), min(math.ceil(place(s["low"])), rot - 1)
        for i, x in enumerate(w):
            keep = 1 - min(max((i - first) / ((last - first) or 0.001), 0), 1)
            w[i] = x * keep + x / f * (1 - keep)
    if kind == "banded":
        for i, x in enumerate(w):
            wave = 2 * math.pi / x
            if wave > old / s["low"]:
                w[i] = x / f
            elif wave >= old / s["high"]:
                mix = (old / wave - s["low"]) / (s["high"] - s["low"])
                w[i] = (1 - mix) * x / f + mix * x
    return torch.tensor(w, dtype=torch.float64), (0.1 * math.log(f) + 1 if kind == "yarn" else 1.0)
