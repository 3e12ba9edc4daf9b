"""Latent caches on the GPU: write and read-back against the layout and the
quantization rules, absorbed and expanded attention against the formulas in
64 bits, at the sizes, masks and values where they can go wrong."""
import math

import pytest
import torch

from _helpers import guarded, kvq
from _latent import MODES, P, R, Batch, compare, decode, empty_cache, four, identity_table, row_bytes

pytestmark = pytest.mark.gpu
F16, F32 = torch.float16, torch.float32


# ---------------------------------------------------------------- write and read
def _codes(x, mode, scale):
    """The stored value of fp32 rows x, by the rules, IEEE operation by operation (CPU)."""
    def fp8(y): return y.clamp(-448, 448).to(torch.float8_e4m3fn).float()  # noqa: E704
    if mode == "fp8_per_tensor":
        return fp8(x / scale).double() * float(scale)
    if not four(mode):
        top = 127.0 if mode.startswith("int8") else 448.0
        s = x.abs().amax(-1, keepdim=True).clamp_min(1e-8) / torch.tensor(top)
        y = x / s
        return (torch.round(y).clamp(-127, 127) if top == 127.0 else fp8(y)).double() * s.double()
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
    b = x.unflatten(-1, (-1, 16))

    def coded(div):
        sb = fp8(b.abs().amax(-1, keepdim=True) / (torch.tensor(div) * scale))
        den = sb * scale
        y = torch.where(den > 0, b / torch.where(den > 0, den, torch.tensor(1.0)), torch.tensor(0.0))
        d = (y.abs().unsqueeze(-1) - grid).abs()
        lo = d.argmin(-1)  # of two equally near, the lower index; ties go to the even code
        hi = (lo + 1).clamp(max=7)
        tie = d.gather(-1, lo.unsqueeze(-1)) == d.gather(-1, hi.unsqueeze(-1))
        code = torch.where(tie.squeeze(-1) & (lo % 2 == 1), hi, lo)
        return torch.sign(y) * grid[code], sb, den
    v6, s6, d6 = coded(6.0)
    if mode == "nvfp4":
        return (v6.double() * s6.double() * float(scale)).flatten(-2)
    v4, s4, d4 = coded(4.0)

    def sse(v, den):
        e = (b - v * den) ** 2
        while e.shape[-1] > 1:
            e = e[..., 0::2] + e[..., 1::2]
        return e
    pick = sse(v4, d4) < sse(v6, d6)
    return (torch.where(pick, v4.double() * s4.double(), v6.double() * s6.double()) * float(scale)).flatten(-2)


def _turned(y, ang, interleaved):
    cos, sin = ang[:, None, :R // 2], ang[:, None, R // 2:]
    z = torch.empty_like(y)
    a, b = (y[..., 0::2], y[..., 1::2]) if interleaved else (y[..., :R // 2], y[..., R // 2:])
    za, zb = a * cos - b * sin, b * cos + a * sin
    if interleaved:
        z[..., 0::2], z[..., 1::2] = za, zb
    else:
        z[..., :R // 2], z[..., R // 2:] = za, zb
    return z


@pytest.mark.parametrize("io", [F16, F32], ids=["f16", "f32"])
@pytest.mark.parametrize("L", [256, 512])
@pytest.mark.parametrize("mode", MODES)
def test_write(mode, L, io):
    """Every output is the correctly rounded value, the pool holds the codes of the rounded rows, and the read-back gives
    what they stand for; skipped and flagged tokens leave everything as it was."""
    K = kvq()
    g = torch.Generator().manual_seed(3)
    T, H = 77, 5
    cache = empty_cache(mode, L, 8, io)
    before = cache.pool.clone()
    wide = torch.randn(T, L + R + 8, generator=g)
    wide[7] *= 1e-6
    wide[9] *= 300.0
    wide[11, :L] = 0.0
    q = torch.randn(T, H, 128 + R, generator=g)
    wide, q = wide.to(io).cuda(), q.to(io).cuda()
    w = (1 + 0.3 * torch.randn(L, generator=g)).to(io)
    pos = torch.randint(0, 300, (T,), generator=g).int()
    pos[5], pos[6] = 300, -1  # skipped and flagged
    ang = torch.randn(300, R // 2, generator=g).double() * 50
    table = torch.cat([ang.cos(), ang.sin()], 1).float()
    slots = torch.randperm(8 * P, generator=g)[:T].int()
    slots[0], slots[1] = -3, 8 * P  # not written; past the pool
    q_out = guarded((T, H, L + R), io, fill=7.0, name="q_out")
    lat, kro = guarded((T, L), io, fill=7.0, name="latent_out"), guarded((T, R), io, fill=7.0, name="k_rope_out")
    inter = L == 256
    K.kvq_latent_write(cache, wide[:, 8:8 + L], wide[:, 8 + L:], pos.cuda(), table.cuda(), slot_mapping=slots.cuda(),
                       q_rope=q[..., 128:], q_rope_out=q_out[..., L:], latent_weight=w.cuda(), latent_out=lat, k_rope_out=kro,
                       eps=1e-5, interleaved=inter)
    assert K.kvq_latent_read_errors(cache) == 0x1 | 0x80
    ok = torch.ones(T, dtype=torch.bool)
    ok[5] = ok[6] = False
    x = wide[:, 8:8 + L].double().cpu()
    want = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + torch.tensor(1e-5).double()) * w.double()
    a = table.double()[pos.long().clamp(0, 299)]
    for got, ref in ((lat, want), (kro, _turned(wide[:, None, 8 + L:].double().cpu(), a, inter)[:, 0]),
                     (q_out[..., L:], _turned(q[..., 128:].double().cpu(), a, inter))):
        assert torch.equal(got.cpu()[ok], ref.to(io)[ok])  # (ties of a 64-bit value's rounding do not occur here)
        assert bool((got.cpu()[~ok] == 7.0).all())
    assert bool((q_out[..., :L] == 7.0).all())
    # the pool
    put = ok.clone()
    put[0] = put[1] = False
    c, r = decode(cache.pool, mode, L, slots[put])
    st = cache.pool[16:20].cpu().view(torch.float32)
    assert torch.equal(c, _codes(lat.cpu().float(), mode, st)[put])
    assert torch.equal(r, kro.cpu().half().double()[put])
    used = torch.zeros(8 * P, dtype=torch.bool)
    used[slots[put].long()] = True
    left = torch.nonzero(~used).flatten().int()
    page = row_bytes(mode, L) * P
    rows = [(cache.pool, before)]
    codes = L // 2 if four(mode) else L
    for now, was in rows:  # slots that nothing was written to keep their bytes
        for s in left.tolist():
            at = 256 + s // P * page + s % P * codes
            assert torch.equal(now[at:at + codes], was[at:at + codes])
    # read-back, one slot twice, skipped and flagged ones
    ask = torch.cat([slots[put], slots[put][:1], torch.tensor([-1, 8 * P], dtype=torch.int32)])
    back, rope = guarded((len(ask), L), io, fill=7.0, name="back"), guarded((len(ask), R), io, fill=7.0, name="rope")
    K.kvq_latent_read(cache, ask.cuda(), back, rope)
    assert K.kvq_latent_read_errors(cache) == 0x1
    assert bool((back[-2:] == 7.0).all()) and bool((rope[-2:] == 7.0).all())
    c, r = decode(cache.pool, mode, L, ask[:-2])
    assert torch.equal(rope.cpu()[:-2].double(), r)
    half = torch.finfo(io).eps / 2
    # one rounding in fp32 and one to io; fp16 results under 2^-14 in steps of 2^-24
    assert bool(((back.cpu()[:-2].double() - c).abs() <= c.abs() * (half + 2.0 ** -24) * 1.001 + (2.0 ** -25 if io == F16 else 0)).all())
    one_side = guarded((len(ask), R), F32, fill=7.0, name="rope32")
    K.kvq_latent_read(cache, ask.cuda(), None, one_side)
    assert torch.equal(one_side.cpu()[:-2].double(), r)
    K.kvq_latent_read_errors(cache)


@pytest.mark.parametrize("T", [1, 8, 9, 33])
def test_write_sizes_and_places(T):
    """No weight, no queries, no slots; outputs over their inputs."""
    K = kvq()
    cache = empty_cache("int8_per_token_head", 512, 4)
    before = cache.pool.clone()
    x, kr = torch.randn(T, 512).half().cuda(), torch.randn(T, R).half().cuda()
    ang = torch.randn(64, R // 2).double()
    table = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
    pos = torch.arange(T).int() % 64
    want = _turned(kr.double().cpu()[:, None], table.double().cpu()[pos.long()], False)[:, 0].half()
    x0 = x.clone()
    K.kvq_latent_write(cache, x, kr, pos.cuda(), table, latent_out=x, k_rope_out=kr)
    assert torch.equal(kr.cpu(), want) and torch.equal(x, x0) and torch.equal(cache.pool, before)
    q = torch.randn(T, 3, R).half().cuda()
    want = _turned(q.double().cpu(), table.double().cpu()[pos.long()], False).half()
    K.kvq_latent_write(cache, x, kr, pos.cuda(), table, q_rope=q, q_rope_out=q)
    assert torch.equal(q.cpu(), want) and torch.equal(cache.pool, before)


@pytest.mark.parametrize("size", [1e-30, 1e30])
def test_write_range_f32(size):
    """fp32 rows whose squares leave fp32's range are normed all the same."""
    K = kvq()
    cache = empty_cache("fp8_per_token_head", 512, 4, F32)
    x = (torch.randn(3, 512) * size).cuda()
    out = torch.empty_like(x)
    w = torch.ones(512).cuda()
    K.kvq_latent_write(cache, x, torch.zeros(3, R).cuda(), torch.zeros(3, dtype=torch.int32).cuda(), identity_table(1),
                       latent_weight=w, latent_out=out, eps=0.0)
    d = x.double()
    assert torch.equal(out, (d / d.square().mean(-1, keepdim=True).sqrt()).float())


def test_scale_from_amax():
    K = kvq()
    for mode, top in (("fp8_per_tensor", 448.0), ("nvfp4", 2688.0)):
        cache = empty_cache(mode, 256, 1)
        K.kvq_latent_set_scale_from_amax(cache, torch.tensor([3.5]).cuda())
        assert cache.pool[16:20].cpu().view(F32).item() == (torch.tensor(3.5) / top).item()


# ---------------------------------------------------------------- absorbed attention
RAGGED = dict(m=[1, 0, 3, 5, 2, 4], n=[1, 40, 3, 130, 0, 2])       # a first token, no queries, whole prompts, none cached
LONG = dict(m=[1, 2, 1], n=[385, 700, 16])
CHUNK = dict(m=[37, 150], n=[200, 150])


def check(b, out_dtype=None, **kw):
    out, lse = b.run(out_dtype, **kw)
    ref, rl, tol, ltol = b.reference(kw.get("causal", True), kw.get("q"))
    rows = sum(b.m)
    tensor_cores = b.io == F16 and (out_dtype or F16) == F16
    worst = compare(out[:rows], ref, tol, b.mass if tensor_cores else None)
    empty = rl == -math.inf
    assert bool((lse[:rows][empty] == -math.inf).all()) and bool((out[:rows][empty] == 0).all())
    assert bool(((lse[:rows].double() - rl).abs()[~empty] <= ltol[~empty]).all())
    assert bool(torch.isnan(out[rows:]).all()) and bool(torch.isnan(lse[rows:]).all())  # rows of no sequence: untouched
    return worst


@pytest.mark.parametrize("causal", [True, False], ids=["causal", "all"])
@pytest.mark.parametrize("heads", [1, 5, 20, 64])
@pytest.mark.parametrize("L", [256, 512])
@pytest.mark.parametrize("mode", MODES)
def test_attention_ragged(mode, L, heads, causal):
    check(Batch(mode, L, heads=heads, seed=heads, extra_rows=3, **RAGGED), causal=causal)


@pytest.mark.parametrize("heads,lens", [(16, LONG), (40, LONG), (128, LONG), (3, CHUNK), (20, CHUNK)])
@pytest.mark.parametrize("mode,L", [("int8_per_token_head", 512), ("nvfp4", 512), ("fp8_per_token_head", 256),
                                    ("fp8_per_tensor", 512)])
def test_attention_lengths(mode, L, heads, lens):
    check(Batch(mode, L, heads=heads, seed=1, **lens))


@pytest.mark.parametrize("max_n", [700, 5000, 100000])
def test_attention_parts(max_n):
    """Bounds far above the lengths: more parts than tiles, most of them empty."""
    b = Batch("int8_per_token_head", 512, heads=20, seed=2, **LONG)
    check(b, max_n=max_n)
    assert b.splits > 1


@pytest.mark.parametrize("heads", [16, 32, 64, 100])
@pytest.mark.parametrize("L", [256, 512])
def test_attention_many_tiles(L, heads):
    """One range of many tiles in one part: the ring, the references and the score buffers go round."""
    b = Batch("fp8_per_token_head", L, [1] * 160, [1500] + [3] * 159, heads, seed=5)
    check(b)


@pytest.mark.parametrize("io,out", [(F32, F32), (F32, F16), (F16, F32)], ids=["f32", "f32_f16", "f16_f32"])
@pytest.mark.parametrize("mode,L", [("int8_per_token_head", 512), ("nvfp4", 256), ("fp8_per_tensor", 256), ("fp8_per_token_head", 512)])
def test_attention_fp32(mode, L, io, out):
    b = Batch(mode, L, heads=5, io=io, seed=4, extra_rows=2, **RAGGED)
    check(b, out)
    check(b, out, causal=False)
    check(Batch(mode, L, heads=3, io=io, seed=6, **LONG), out, max_n=3000)


@pytest.mark.parametrize("q_size", [0.0, 1e-4, 30.0])
@pytest.mark.parametrize("spread", [None, 4.0])
def test_attention_values(q_size, spread):
    """Scores from none to hundreds, tokens whose scales lie far apart: references move, in long ranges too."""
    for mode in ("int8_per_token_head", "fp8_per_token_head"):
        check(Batch(mode, 512, [2, 1], [300, 900], 20, seed=7, q_size=q_size, spread=spread))


def test_attention_rising():
    """Scores that rise from tile to tile by more than the slack: the accumulator is rescaled at each."""
    b = Batch("int8_per_token_head", 512, [1], [1300], 16, seed=8)
    K = kvq()
    c = torch.randn(1300, 512) * torch.linspace(0.2, 12, 1300)[:, None]
    c[:, 0] = torch.linspace(0, 400, 1300)
    K.kvq_latent_write(b.cache, c.half().cuda(), torch.randn(1300, R).half().cuda(), torch.zeros(1300, dtype=torch.int32).cuda(),
                       identity_table(1), slot_mapping=b.slots.cuda())
    b.q[:, :, 0] = 3.0
    check(b)


def test_attention_bad_numbers():
    """NaN and infinite queries make their own rows NaN and no others."""
    b = Batch("nvfp4", 512, [2, 1], [200, 50], 20, seed=9)
    q = b.q.clone()
    q[0, 3, 17], q[1, 5, 540], q[2, 19, 0] = float("nan"), float("inf"), float("-inf")
    out, lse = b.run(q=q)
    bad = torch.zeros(3, 20, dtype=torch.bool)
    bad[0, 3] = bad[1, 5] = bad[2, 19] = True
    assert bool(torch.isnan(out[bad]).all()) and bool(torch.isnan(lse[bad]).all())
    ref, rl, tol, _ = b.reference()
    compare(out[~bad], ref[~bad], tol[~bad], b.mass[~bad])


def test_attention_missing_pages_and_lens():
    """A page id outside the pool drops its tokens; a length over its bound is cut; bad query ranges have no rows."""
    b = Batch("int8_per_token_head", 512, [2, 3], [300, 90], 20, seed=10)
    b.table[0, 3], b.table[1, 1] = 10 ** 6, -1
    out, lse = b.run(check=0x2)
    ref, rl, tol, ltol = b.reference(drop=[(0, 3), (1, 1)])
    compare(out, ref, tol, b.mass)
    assert bool(((lse.double() - rl).abs() <= ltol).all())
    b = Batch("int8_per_token_head", 512, [2, 3], [300, 90], 20, seed=10)
    b.cu = torch.tensor([0, 2, 9], dtype=torch.int32)  # past the batch
    out, _ = b.run(check=0x100)
    assert bool(torch.isnan(out[2:]).all()) and not bool(torch.isnan(out[:2]).any())
    b.cu = torch.tensor([0, 2, 5], dtype=torch.int32)
    out, _ = b.run(max_q=2, check=0x100)  # a chunk over its bound
    assert bool(torch.isnan(out[2:]).all()) and not bool(torch.isnan(out[:2]).any())
    full, _ = b.run()
    b.n = [300, 1000]
    b.table = b.table[:, :19]
    out, _ = b.run(max_n=300, check=0x2 | 0x8)  # cut to 300 tokens, of which pages are missing
    assert torch.equal(out[:2], full[:2])


def test_attention_unwritten_slots():
    """Bytes behind a sequence's end, NaN codes among them, have no effect."""
    for mode in ("fp8_per_token_head", "nvfp4"):
        b = Batch(mode, 512, [1, 2], [131, 17], 20, seed=11)
        first, _ = b.run()
        page = row_bytes(mode, 512) * P
        for seq, n in ((0, 131), (1, 17)):
            p, t = int(b.table[seq, n // P]), n % P
            body = b.cache.pool[256 + p * page:256 + (p + 1) * page]
            codes = 256 if four(mode) else 512
            body[t * codes:P * codes] = 0x7F
            body[P * codes + t * 2 * R:P * codes + P * 2 * R] = 0xFF
            at = P * codes + P * 2 * R
            step = 32 if four(mode) else 4
            body[at + t * step:at + P * step] = 0xFF
        again, _ = b.run()
        assert torch.equal(first, again)


def test_attention_streams_and_graphs():
    """Another stream; two captured graphs with a workspace each, replayed on new lengths and queries, then side by side."""
    K = kvq()
    b = Batch("fp8_per_token_head", 512, [1, 1], [400, 900], 20, seed=12)
    want, _ = b.run()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got, _ = b.run()
    assert torch.equal(got, want)
    got, _ = b.run(stream=side)
    assert torch.equal(got, want)
    graphs, cu, table = [], b.cu.cuda(), b.table.cuda()
    for _ in range(2):
        q, n = b.q.cuda().clone(), torch.tensor(b.n, dtype=torch.int32).cuda()
        out = torch.zeros(2, 20, 512, dtype=F16, device="cuda")
        parts, ws = K.kvq_latent_plan(b.cache, 2, 2, 20, max_q_len=1, max_seq_len=900)
        assert parts > 1
        work = torch.empty(ws, dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            K.kvq_latent_attention(b.cache, q, cu, table, n, out, max_q_len=1, max_seq_len=900, softmax_scale=b.scale, workspace=work)
        graphs.append((graph, q, n, out, work))
    for graph, _, _, out, _ in graphs:
        graph.replay()
        assert torch.equal(out.cpu(), want)
    q2 = torch.randn_like(b.q)
    want2, _ = b.run(q=q2)
    graphs[1][1].copy_(q2.cuda())
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(side):
            graphs[0][0].replay()
        graphs[1][0].replay()
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][3].cpu(), want) and torch.equal(graphs[1][3].cpu(), want2)


def test_attention_repeats_bit_for_bit():
    b = Batch("nvfp4", 512, [3, 40], [900, 300], 40, seed=13)
    first, l1 = b.run(max_n=4000)
    for _ in range(3):
        again, l2 = b.run(max_n=4000)
        assert torch.equal(first, again) and torch.equal(l1, l2)


def test_together():
    """Write, attend and read as a layer uses them: a prompt chunk, then decode steps, equal the formula over the read rows."""
    K = kvq()
    g = torch.Generator().manual_seed(14)
    L, H, cache = 512, 20, empty_cache("fp8_per_token_head", 512, 20)
    ang = torch.arange(400, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(R // 2, dtype=torch.float64) / (R // 2))
    cs = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
    table = torch.randperm(20, generator=g).int()[None].cuda()
    w = torch.ones(L).half().cuda()
    at = 0
    for m in (150, 1, 1, 7):
        pos = torch.arange(at, at + m)
        slots = table.cpu()[0, pos // P] * P + pos % P
        ckr = torch.randn(m, L + R, generator=g).half().cuda()
        q = torch.zeros(m, H, L + R).half().cuda()
        q[..., :L] = 0.6 * torch.randn(m, H, L, generator=g).half().cuda()
        qr = torch.randn(m, H, 128 + R, generator=g).half().cuda()
        K.kvq_latent_write(cache, ckr[:, :L], ckr[:, L:], pos.int().cuda(), cs, slot_mapping=slots.int().cuda(), q_rope=qr[..., 128:],
                           q_rope_out=q[..., L:], latent_weight=w)
        at += m
        _, ws = K.kvq_latent_plan(cache, m, 1, H, max_q_len=m, max_seq_len=at)
        out, work = torch.empty(m, H, L).half().cuda(), torch.empty(max(ws, 16), dtype=torch.uint8, device="cuda")
        K.kvq_latent_attention(cache, q, torch.tensor([0, m]).int().cuda(), table, torch.tensor([at]).int().cuda(), out, max_q_len=m,
                               max_seq_len=at, softmax_scale=192.0 ** -0.5, workspace=work)
        all_slots = (table.cpu()[0, torch.arange(at) // P] * P + torch.arange(at) % P).int().cuda()
        c, kr = torch.empty(at, L, device="cuda"), torch.empty(at, R, device="cuda")
        K.kvq_latent_read(cache, all_slots, c, kr)
        assert K.kvq_latent_read_errors(cache) == 0
        k = torch.cat([c, kr], 1).double()
        s = torch.einsum("ihd,td->iht", q.double(), k) * 192.0 ** -0.5
        s = s.masked_fill(torch.arange(at, device="cuda") > pos.cuda()[:, None, None], -math.inf)
        p = torch.softmax(s, -1)
        ref, mass = torch.einsum("iht,td->ihd", p, c.double()), torch.einsum("iht,td->ihd", p, c.double().abs())
        # weights and outputs by half a step of fp16 each; scores as in Batch.reference, sum |q k| here below 60
        assert bool(((out.double() - ref).abs() <= 2.0 ** -11 * (mass + ref.abs()) + mass * 2 * 40 * 2.0 ** -23 * 60 + 2.0 ** -25).all())


# ---------------------------------------------------------------- expanded attention
class Prompt:
    def __init__(self, m, n, heads, io=F16, seed=0, size=1.0, extra=0):
        g = torch.Generator().manual_seed(seed)
        self.m, self.n, self.heads, self.io = m, n, heads, io
        self.q = (size * torch.randn(sum(m) + extra, heads, 128 + R, generator=g)).to(io)
        self.kv = torch.randn(sum(n) + extra, heads, 256, generator=g).to(io)
        self.kr = (1.5 * torch.randn(sum(n) + extra, R + 8, generator=g)).to(io)
        self.cu = torch.tensor([sum(m[:b]) for b in range(len(m) + 1)], dtype=torch.int32)
        self.cuk = torch.tensor([sum(n[:b]) for b in range(len(n) + 1)], dtype=torch.int32)
        self.cache = empty_cache("fp8_per_token_head", 512, 1, io)

    def run(self, out_dtype=None, causal=True, check=0, max_q=None, max_k=None, stream=None):
        K = kvq()
        out = guarded((self.q.shape[0], self.heads, 128), out_dtype or self.io, fill=float("nan"), name="out")
        lse = guarded((self.q.shape[0], self.heads), F32, fill=float("nan"), name="lse")
        kv = self.kv.cuda()
        K.kvq_latent_prompt_attention(self.cache, self.q.cuda(), kv[..., :128], self.kr.cuda()[:, :R], kv[..., 128:], self.cu.cuda(),
                                      self.cuk.cuda(), out, max_q_len=max_q or max(max(self.m), 1),
                                      max_k_len=max_k or max(max(self.n), 1), causal=causal, lse=lse, stream=stream)
        torch.cuda.synchronize()
        assert K.kvq_latent_read_errors(self.cache) == check
        return out.cpu(), lse.cpu()

    def check(self, out_dtype=None, causal=True, **kw):
        """Tolerances as in Batch.reference, of 192-term scores."""
        out, lse = self.run(out_dtype, causal, **kw)
        exact = self.io == F16
        half = torch.finfo(out.dtype).eps / 2
        tensor_cores = exact and out.dtype == F16
        for b in range(len(self.m)):
            n, m = self.n[b], self.m[b]
            r, k0 = int(self.cu[b]), int(self.cuk[b])
            q = self.q[r:r + m].double()
            k = torch.cat([self.kv[k0:k0 + n, :, :128].double(), self.kr[k0:k0 + n, None, :R].double().expand(-1, self.heads, -1)], -1)
            v = self.kv[k0:k0 + n, :, 128:].double()
            see = torch.arange(n) <= (torch.arange(n - m, n) if causal else torch.full((m,), n - 1))[:, None, None]
            s = torch.einsum("ihd,thd->iht", q, k) * 192.0 ** -0.5
            see = see.expand_as(s)
            s = s.masked_fill(~see, -math.inf)
            ls = torch.logsumexp(s, -1) if n else torch.full((m, self.heads), -math.inf, dtype=torch.float64)
            w = torch.where(see, torch.exp(s - torch.where(ls == -math.inf, 0.0, ls).unsqueeze(-1)), 0.0)
            ref, mass = torch.einsum("iht,thd->ihd", w, v), torch.einsum("iht,thd->ihd", w, v.abs())
            size = torch.einsum("ihd,thd->iht", q.abs(), k.abs()) * 192.0 ** -0.5
            size = torch.where(see, size, 0.0).amax(-1) if n else torch.zeros(m, self.heads, dtype=torch.float64)
            d = (16 * 2.0 ** -23 if exact else 196 * 2.0 ** -24) * size
            steps = n / 16 * 2.0 ** -23 if exact else (n + 8) * 2.0 ** -24
            tol = mass * (2 * d.unsqueeze(-1) + 2.0 ** -21 + steps + (2.0 ** -11 if tensor_cores else 0)) * (1 + half) \
                + half * ref.abs() + (2.0 ** -25 if out.dtype == F16 else 1e-30)
            assert bool(((out[r:r + m].double() - ref).abs() <= tol).all()), b
            none = ls == -math.inf
            assert bool((lse[r:r + m][none] == -math.inf).all())
            lt = d + 2.0 ** -21 + 2.0 ** -22 * torch.where(none, 0.0, ls).abs()
            assert bool(((lse[r:r + m].double() - ls).abs()[~none] <= lt[~none]).all())
        rows = sum(self.m)
        assert bool(torch.isnan(out[rows:]).all()) and bool(torch.isnan(lse[rows:]).all())


@pytest.mark.parametrize("causal", [True, False], ids=["causal", "all"])
@pytest.mark.parametrize("io,out", [(F16, F16), (F32, F32), (F16, F32)], ids=["f16", "f32", "f16_f32"])
@pytest.mark.parametrize("m,n", [([1, 0, 3, 5, 2, 4], [1, 40, 3, 130, 0, 2]), ([129, 300], [129, 450]), ([1, 40], [700, 1000])],
                         ids=["ragged", "prompts", "tails"])
def test_prompt(m, n, io, out, causal):
    Prompt(m, n, 3, io, seed=1, extra=2).check(out, causal)


@pytest.mark.parametrize("m,n,heads", [([1000], [1000], 2), ([257, 64, 513], [257, 900, 600], 5), ([128], [128], 1), ([2], [2], 128)])
def test_prompt_lengths(m, n, heads):
    Prompt(m, n, heads, seed=2).check()


@pytest.mark.parametrize("size", [0.0, 1e-3, 40.0])
def test_prompt_values(size):
    Prompt([200], [500], 4, seed=3, size=size).check()


def test_prompt_bad_numbers_and_ranges():
    p = Prompt([130, 5], [300, 64], 3, seed=4)
    good, _ = p.run()
    p.q[3, 1, 5], p.q[131, 2, 190] = float("nan"), float("inf")
    out, lse = p.run()
    bad = torch.zeros(135, 3, dtype=torch.bool)
    bad[3, 1] = bad[131, 2] = True
    assert bool(torch.isnan(out[bad]).all()) and bool(torch.isnan(lse[bad]).all()) and torch.equal(out[~bad], good[~bad])
    p = Prompt([130, 5], [300, 64], 3, seed=4)
    for cuk in ([0, 300, 365], [0, 300, 299], [-1, 300, 364]):
        p.cuk = torch.tensor(cuk, dtype=torch.int32)
        out, _ = p.run(check=0x100)
        skipped = slice(0, 130) if cuk[0] < 0 else slice(130, 135)
        assert bool(torch.isnan(out[skipped]).all())
        kept = torch.ones(135, dtype=torch.bool)
        kept[skipped] = False
        assert torch.equal(out[kept], good[kept])
    p.cuk = torch.tensor([0, 300, 364], dtype=torch.int32)
    out, _ = p.run(check=0x100, max_k=299)
    assert bool(torch.isnan(out[:130]).all()) and torch.equal(out[130:], good[130:])


def test_prompt_streams_and_graphs():
    K = kvq()
    p = Prompt([130, 5], [300, 64], 3, seed=5)
    want, _ = p.run()
    side = torch.cuda.Stream()
    got, _ = p.run(stream=side)
    assert torch.equal(got, want)
    q, kv, kr, cu, cuk = p.q.cuda(), p.kv.cuda(), p.kr.cuda(), p.cu.cuda(), p.cuk.cuda()
    out = torch.zeros(135, 3, 128, dtype=F16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        K.kvq_latent_prompt_attention(p.cache, q, kv[..., :128], kr[:, :R], kv[..., 128:], cu, cuk, out, max_q_len=130, max_k_len=300)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), want)


@pytest.mark.parametrize("max_k", [20000, 70000])
def test_prompt_head_groups(max_k):
    """Bounds for which heads run in groups (of three and two of five; one by one), over ranges of many tiles."""
    Prompt([300, 40, 1], [2500, 40, 2200], 5, seed=9, extra=1).check(max_k=max_k)
    Prompt([300, 40], [1500, 700], 5, seed=10).check(causal=False, max_k=max_k)


def test_prompt_rows_that_see_nothing():
    """Tiles of rows without a key beside tiles with many: their zeros are not written over by copies in flight."""
    p = Prompt([2, 300] * 20, [0, 300] * 20, 8, seed=6)
    for _ in range(5):
        out, lse = p.run()
        none = torch.cat([torch.arange(302 * i, 302 * i + 2) for i in range(20)])
        assert bool((out[none] == 0).all()) and bool((lse[none] == -math.inf).all())


def test_prompt_without_keys():
    p = Prompt([3, 2], [0, 0], 2, seed=7)
    out, lse = p.run()
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


# ---------------------------------------------------------------- calls that the documentation allows
def test_ranges_that_repeat():
    """Chunk ranges that are no ascending list: the backward ones are flagged, and nothing is written outside the buffers."""
    K = kvq()
    b = Batch("fp8_per_token_head", 512, [1] * 60, [300] * 60, 16, seed=15)
    q, out = b.q[:1].cuda(), guarded((1, 16, 512), F16, fill=float("nan"), name="out")
    cu = torch.tensor([0, 1] * 30 + [0], dtype=torch.int32).cuda()
    _, ws = K.kvq_latent_plan(b.cache, 1, 60, 16, max_q_len=1, max_seq_len=300)
    work = guarded(max(ws, 16), torch.uint8, fill=0xFF, name="workspace")
    K.kvq_latent_attention(b.cache, q, cu, b.table.cuda(), torch.full((60,), 300, dtype=torch.int32).cuda(), out, max_q_len=1,
                           max_seq_len=300, softmax_scale=b.scale, workspace=work)
    torch.cuda.synchronize()
    assert K.kvq_latent_read_errors(b.cache) == 0x100


def test_many_sequences():
    """More sequences than a plan of parts takes, most of them short, and a batch of one long one."""
    n = [(37 * b) % 50 for b in range(700)]
    check(Batch("int8_per_token_head", 256, [1] * 700, n, 2, seed=16))
    check(Batch("nvfp4", 512, [1], [20000], 3, seed=17))


def test_unequal_lengths():
    """One long sequence among short ones, with and without split ranges: parts of every size."""
    for heads in (16, 64, 128):
        check(Batch("fp8_per_token_head", 512, [1, 2, 1, 3, 1], [9000, 5, 130, 700, 1], heads, seed=18))


def test_offsets_past_32_bits():
    """Pages beyond four gigabytes of a pool."""
    K = kvq()
    pages = 420000
    cfg = K.make_latent_config(pages, P, 512, R, "fp8_per_token_head", F16)
    pool = torch.empty(K.kvq_latent_bytes(cfg), dtype=torch.uint8, device="cuda")
    assert pool.numel() > 1 << 32
    cache = K.kvq_latent_alloc(cfg, pool)
    n = 200
    table = torch.arange(pages - 13, pages, dtype=torch.int32)[None]
    slots = (table[0, torch.arange(n) // P] * P + torch.arange(n) % P).int().cuda()
    c, kr = torch.randn(n, 512).half().cuda(), torch.randn(n, R).half().cuda()
    K.kvq_latent_write(cache, c, kr, torch.zeros(n, dtype=torch.int32).cuda(), identity_table(1), slot_mapping=slots)
    back, rope = torch.empty_like(c), torch.empty_like(kr)
    K.kvq_latent_read(cache, slots, back, rope)
    assert torch.equal(rope, kr)
    q, out = torch.randn(1, 8, 576).half().cuda(), torch.empty(1, 8, 512).half().cuda()
    _, ws = K.kvq_latent_plan(cache, 1, 1, 8, max_q_len=1, max_seq_len=n)
    K.kvq_latent_attention(cache, q, torch.tensor([0, 1]).int().cuda(), table.cuda(), torch.tensor([n]).int().cuda(), out, max_q_len=1,
                           max_seq_len=n, softmax_scale=0.05, workspace=torch.empty(max(ws, 16), dtype=torch.uint8, device="cuda"))
    assert K.kvq_latent_read_errors(cache) == 0
    k = torch.cat([back, rope], 1).double()  # (fp16 rows of fp8 codes times their scales: 2^-11 of each)
    p = torch.softmax(q.double()[0] @ k.T * 0.05, -1)
    mass = p @ back.double().abs()
    assert bool(((out.double()[0] - p @ back.double()).abs() <= 2.0 ** -11 * 4 * mass + 0.05 * 600 * 4 * 2.0 ** -11 * mass).all())


def test_python_refusals():
    K = kvq()
    b = Batch("fp8_per_token_head", 512, [1], [40], 4, seed=19)
    args = lambda **kw: dict(dict(q=b.q.cuda(), cu=b.cu.cuda(), table=b.table.cuda(), n=torch.tensor([40]).int().cuda(),  # noqa: E731
                                  out=torch.empty(1, 4, 512).half().cuda()), **kw)
    for bad in (dict(q=b.q.float().cuda()), dict(q=b.q.cuda()[..., :512]), dict(cu=b.cu.long().cuda()), dict(cu=b.cu),
                dict(out=torch.empty(1, 4, 576).half().cuda()), dict(out=torch.empty(1, 4, 512).bfloat16().cuda()),
                dict(n=torch.tensor([40, 1]).int().cuda()), dict(table=b.table.cuda()[0])):
        a = args(**bad)
        with pytest.raises((ValueError, K.KVQError)):
            K.kvq_latent_attention(b.cache, a["q"], a["cu"], a["table"], a["n"], a["out"], max_q_len=1, max_seq_len=40, softmax_scale=0.1)
    with pytest.raises(ValueError):
        K.kvq_latent_read(b.cache, torch.zeros(2, dtype=torch.int32).cuda(), torch.empty(3, 512).half().cuda())
    with pytest.raises(ValueError):
        K.kvq_latent_write(b.cache, torch.zeros(512, 2).half().cuda().t(), torch.zeros(2, R).half().cuda(),
                           torch.zeros(2, dtype=torch.int32).cuda(), identity_table(1))
    with pytest.raises(AttributeError):
        K.kvq_decode_attention(b.cache, b.q.cuda(), b.table.cuda(), torch.tensor([40]).int().cuda(), torch.empty(1, 4, 512).half().cuda(),
                               max_seq_len=40, softmax_scale=0.1)
