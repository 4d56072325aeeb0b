"""GPU parity of rotary positions and of the block-scaled 8-bit cache (append,
read back, attention, accumulated weight, eviction) against the plain forms of
b8_reference.py.  Tolerances follow from the roundings that each call makes
and are stated where they are used."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import b8_reference as ref
from hadamard_rotated_bit_fwht_b200 import build, kvq

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    kvq.lib()
    kvq.device_errors()
    yield
    assert kvq.device_errors() == 0


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def rand(seed, *shape, dtype=F32, outliers=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    if outliers:
        x[..., ::37] *= 16.0
    return x.to(dtype).cuda()


def filled(seed, lens, hkv, dim, block, spare=0, unmapped=()):
    """A cache of random codes and scales over a shuffled table; (sequence,
    column) pairs of `unmapped` have no block.  Blocks of no sequence hold NaN
    scales."""
    g = torch.Generator().manual_seed(seed)
    cols = [(n + block - 1) // block for n in lens]
    nb = sum(cols) + spare + 2
    codes = [torch.randint(-127, 128, (nb, hkv, block, dim), generator=g, dtype=torch.int8)
             for _ in "kv"]
    scales = [torch.exp(torch.randn((nb, hkv), generator=g)) / 64 for _ in "kv"]
    perm = torch.randperm(nb, generator=g).int()
    table = torch.full((len(lens), max(cols + [1])), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(cols):
        table[b, :n] = perm[at:at + n]
        at += n
    for p in perm[at:].tolist():
        for s in scales:
            s[p] = math.nan
    for b, col in unmapped:
        table[b, col] = -1 if (b + col) % 2 else nb + 5
    c = kvq.B8Cache.wrap(codes[0].cuda(), scales[0].cuda(), codes[1].cuda(), scales[1].cuda(),
                         table.cuda())
    return c, perm[at:]


# ------------------------------------------------------------------ rope
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,hq,hkv,dim,rot,inter,fused", [
    (1, 4, 1, 64, 64, False, False), (5, 8, 2, 128, 128, True, True),
    (700, 3, 3, 128, 32, False, True), (2500, 4, 1, 256, 64, True, False),
    (33, 1, 1, 16, 16, False, False), (3, 2, 1, 512, 512, True, False),
    (7, 2, 2, 48, 16, False, True)])
def test_rope(dtype, n, hq, hkv, dim, rot, inter, fused):
    x = rand(n + dim, n, hq + 2 * hkv, dim, dtype=dtype)
    q, k = x[:, :hq], x[:, hq:hq + hkv]
    if not fused:
        q, k = q.contiguous(), k.contiguous()
    g = torch.Generator().manual_seed(n)
    pos = torch.randint(0, 1 << 20, (n,), generator=g, dtype=torch.int32)
    pos[0] = 0
    pos[-1] = 2 ** 31 - 1
    if n > 2:
        pos[1] = -5
    r = kvq.Rope.make(rot, interleaved=inter, scaling="yarn", scale=8.0, trained_len=4096)
    for inverse in (False, True):
        got = kvq.rope(q, k, pos.cuda(), r, inverse=inverse)
        for a, b in zip(got, (q, k)):
            want = ref.rotate(b, pos, r.inv_freq, r.factor, inter, inverse)
            # fp32: the angle is off by 2^-25 half turns + its fp64 error (2^31
            # radians keep 2^-21), sincospi by 2 ulp, the three products and
            # sums by half an ulp each, all times |x| <= 6; then one rounding
            tol = 6 * r.factor * 2 * (3.2 * 2 ** -25 + 2 ** -20 * (pos.double() / 2 ** 31).abs()
                                      + 5 * 2 ** -24)[:, None, None]
            tol = tol + want.abs() * torch.finfo(dtype).eps / 2
            assert ((a.double().cpu() - want).abs() <= tol).all()
            assert torch.equal(a[..., rot:], b[..., rot:])
    # in place, and undone again: the same view as input and output
    y = x.clone()
    kvq.rope(y[:, :hq], y[:, hq:hq + hkv], pos.cuda(), r, q_out=y[:, :hq],
             k_out=y[:, hq:hq + hkv])
    fwd = kvq.rope(q, k, pos.cuda(), r)
    assert torch.equal(y[:, :hq], fwd[0]) and torch.equal(y[:, hq:hq + hkv], fwd[1])
    assert torch.equal(y[:, hq + hkv:], x[:, hq + hkv:])


def test_rope_inverse_is_the_gradient():
    """<rope(x), w> = <x, rope_inverse(w)>, and against central differences."""
    n, h, d = 6, 2, 64
    r = kvq.Rope.make(48, interleaved=True, scaling="yarn", scale=4.0, trained_len=2048)
    x, w = rand(1, n, h, d), rand(2, n, h, d)
    pos = ints([0, 1, 17, 999, 32768, 100000])
    f = lambda x: (kvq.rope(x, None, pos, r)[0].double() * w.double()).sum().item()
    grad = kvq.rope(w, None, pos, r, inverse=True)[0]
    # the two sums have 768 terms below 30, each off by 2^-21 relative
    assert abs(f(x) - (x.double() * grad.double()).sum().item()) < 768 * 30 * 2 ** -21
    for i, j, e in ((0, 0, 3), (3, 1, 0), (5, 0, 47), (4, 1, 60)):
        up, dn = x.clone(), x.clone()
        up[i, j, e] += 1.0
        dn[i, j, e] -= 1.0
        # linear in x: the difference is exact but for the roundings of f's
        # few changed terms (below 60, 2^-21 each)
        assert abs((f(up) - f(dn)) / 2 - grad[i, j, e].item()) < 4 * 60 * 2 ** -21


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope_records_gradients(dtype, inverse):
    r = kvq.Rope.make(32, interleaved=inverse, scaling="yarn", scale=4.0, trained_len=2048)
    x, w = rand(181, 7, 6, 64, dtype=dtype), rand(182, 7, 6, 64, dtype=dtype)
    pos = ints([0, 1, 17, 999, 32768, 100000, -3])
    plain = kvq.rope(x[:, :4], x[:, 4:], pos, r, inverse=inverse)
    gq, gk = kvq.rope(w[:, :4], w[:, 4:], pos, r, inverse=not inverse)
    leaf = x.clone().requires_grad_()
    # slices of one projection
    q, k = kvq.rope(leaf[:, :4], leaf[:, 4:], pos, r, inverse=inverse)
    assert torch.equal(q, plain[0]) and torch.equal(k, plain[1])
    torch.autograd.backward((q, k), (w[:, :4], w[:, 4:]))
    assert torch.equal(leaf.grad, torch.cat((gq, gk), 1))
    # one of the two alone, as input or as what is used of the outputs
    q1 = x[:, :4].clone().requires_grad_()
    kvq.rope(q1, None, pos, r, inverse=inverse)[0].backward(w[:, :4])
    assert torch.equal(q1.grad, gq)
    k1 = x[:, 4:].clone().requires_grad_()
    kvq.rope(x[:, :4], k1, pos, r, inverse=inverse)[1].backward(w[:, 4:])
    assert torch.equal(k1.grad, gk)
    both = [x[:, :4].clone().requires_grad_(), x[:, 4:].clone().requires_grad_()]
    kvq.rope(*both, pos, r, inverse=inverse)[1].backward(w[:, 4:])
    assert both[0].grad is None and torch.equal(both[1].grad, gk)
    # a gradient that comes expanded, in batches, on another stream; a second one
    y = x.view(1, 7, 6, 64).clone().requires_grad_()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        kvq.rope(y, None, pos, r, inverse=inverse)[0].sum().backward()
    torch.cuda.current_stream().wait_stream(st)
    ones = torch.ones_like(x)
    assert torch.equal(y.grad[0], kvq.rope(ones, None, pos, r, inverse=not inverse)[0])
    v = w.clone().requires_grad_()
    z = x.clone().requires_grad_()
    g, = torch.autograd.grad(kvq.rope(z, None, pos, r, inverse=inverse)[0], z, v, create_graph=True)
    g.backward(x)
    assert torch.equal(v.grad, kvq.rope(x, None, pos, r, inverse=inverse)[0])
    # nothing is recorded where nothing is asked for, nor through given outputs
    with torch.no_grad():
        assert kvq.rope(leaf, None, pos, r)[0].grad_fn is None
    assert kvq.rope(x, None, pos, r)[0].grad_fn is None
    o = torch.empty_like(x)
    assert kvq.rope(leaf, None, pos, r, q_out=o)[0] is o and o.grad_fn is None


def test_rope_gradient_in_a_captured_step():
    """Forward and backward captured, all of the leaf's uses on the capture's stream
    (torch refuses a capture beside an eager graph of the same leaf on another)."""
    r = kvq.Rope.make(64)
    w, pos = rand(184, 5, 2, 64), ints([0, 5, 9, 100, 7])
    want, _ = kvq.rope(w, None, pos, r, inverse=True)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        x = rand(183, 5, 2, 64).requires_grad_()
        for _ in range(2):
            torch.autograd.grad(kvq.rope(x, None, pos, r)[0], x, w)
        st.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=st):
            got, = torch.autograd.grad(kvq.rope(x, None, pos, r)[0], x, w)
        got.zero_()
        gr.replay()
    st.synchronize()
    assert torch.equal(got, want)


def test_rope_shapes_streams_and_empty():
    r = kvq.Rope.make(64)
    x = rand(3, 2, 5, 4, 64, dtype=BF16)
    pos = ints(list(range(10)))
    a, none = kvq.rope(x, None, pos, r)
    assert none is None and a.shape == x.shape
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    b, _ = kvq.rope(x, None, pos, r, stream=st)
    st.synchronize()
    assert torch.equal(a, b)
    e, _ = kvq.rope(x[:0], None, pos[:0], r)
    assert e.shape == (0, 5, 4, 64)
    with pytest.raises(ValueError):
        kvq.rope(x, None, pos[:9], r)
    with pytest.raises(ValueError):
        kvq.rope(x, None, pos.long(), r)
    with pytest.raises(TypeError):
        kvq.rope(x.half(), None, pos, r)
    with pytest.raises(ValueError):
        kvq.rope(x.cpu(), None, pos, r)


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim,block,hkv,start,new", [
    (128, 16, 2, [5, 0, 31], [1, 1, 1]), (64, 32, 1, [0, 7, 64, 3], [40, 100, 0, 33]),
    (256, 64, 3, [63, 10], [130, 2]), (128, 256, 1, [0, 255, 700], [256, 300, 1]),
    (256, 256, 2, [17], [700]), (64, 128, 4, [-3, 120], [9, 9])])
def test_append_and_gather(dtype, dim, block, hkv, start, new):
    batch, t_new = len(start), max(new)
    c, _ = filled(dim + block, [max(s + n, 1) for s, n in zip(start, new)], hkv, dim, block)
    x = rand(7, batch, t_new, 3 * hkv, dim, dtype=dtype, outliers=True)
    k, v = x[:, :, :hkv], x[:, :, hkv:2 * hkv]
    x[0, 0, 0] = 0  # an empty row
    before = ref.Cache(c)
    kvq.b8_append(c, k, v, ints(start), new_lens=ints(new))
    want = before
    for b in range(batch):
        want.append(b, start[b], k[b, :new[b]].float().cpu(), v[b, :new[b]].float().cpu())
    # the fp32 operations are pinned: bit-exact, other rows untouched
    for w, codes, scales in (("k", c.k_codes, c.k_scales), ("v", c.v_codes, c.v_scales)):
        assert torch.equal(codes.cpu(), want.codes[w])
        assert torch.equal(scales.cpu().view(torch.int32), want.scales[w].view(torch.int32))
    ends = [max(s + n, 0) for s, n in zip(start, new)]
    first = [max(e - 3, -1) for e in ends]
    count = max(e - f for e, f in zip(ends, first)) + 2
    for dt in (BF16, F32):
        gk, gv = kvq.b8_gather(c, ints(first), ints(ends), count, dt)
        for w, g in (("k", gk), ("v", gv)):
            for b in range(batch):
                val, _ = want.values(w, b, ends[b])
                for i in range(count):
                    t = first[b] + i
                    row = val[:, t].float().to(dt) if 0 <= t < ends[b] else torch.zeros(hkv, dim)
                    assert torch.equal(g[b, i].cpu().float(), row.float())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim,block", [(64, 256), (128, 128), (256, 64), (256, 256)])
def test_append_of_every_length(dtype, dim, block):
    """Each number of new rows has its own share of shared memory: all of them up to
    a block, as one append and as one of a longer padded batch."""
    k, v = rand(197, 1, block, 1, dim, dtype=dtype), rand(198, 1, block, 1, dim, dtype=dtype)
    c, d = (kvq.B8Cache.contiguous(1, 1, block, dim, block) for _ in "cd")
    for n in range(1, block + 1):
        kvq.b8_append(c, k[:, :n], v[:, :n], ints([0]))
        kvq.b8_append(d, k, v, ints([0]), new_lens=ints([n]))
        assert torch.equal(c.k_scales, d.k_scales) and torch.equal(c.v_scales, d.v_scales), n
        assert torch.equal(c.k_codes[:, :, :n], d.k_codes[:, :, :n]), n
        assert torch.equal(c.v_codes[:, :, :n], d.v_codes[:, :, :n]), n


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_append_of_48_kilobytes_first(dtype):
    """33 to 48 rows of 256 dims take 48 KB of shared memory: as the first call of a
    process, before a larger one has asked for more than the default."""
    code = f"""
import torch
from hadamard_rotated_bit_fwht_b200 import kvq
for n in (33, 40, 48):
    c = kvq.B8Cache.contiguous(1, 1, 64, 256, 64)
    x = torch.ones((1, n, 1, 256), dtype=torch.{dtype}, device="cuda")
    kvq.b8_append(c, x, x, torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert (c.k_codes[0, 0, :n] == 127).all() and not c.k_codes[0, 0, n:].any()
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("own_positions", [False, True])
def test_append_with_rope(inter, own_positions):
    batch, t_new, hkv, dim, block = 2, 70, 2, 128, 32
    start, new = [10, 50], [70, 45]
    r = kvq.Rope.make(64, interleaved=inter)
    k, v = rand(11, batch, t_new, hkv, dim), rand(12, batch, t_new, hkv, dim)
    c, _ = filled(13, [80, 95], hkv, dim, block)
    c.k_scales.mul_(1e-3)
    want = ref.Cache(c)
    pos = torch.stack([torch.arange(t_new, dtype=torch.int32) * 3 + s for s in start])
    if not own_positions:
        pos = torch.stack([torch.arange(t_new, dtype=torch.int32) + s for s in start])
    kvq.b8_append(c, k, v, ints(start), new_lens=ints(new), rope=r,
                  positions=pos.cuda() if own_positions else None)
    for b in range(batch):
        kr = ref.rotate(k[b, :new[b]], pos[b, :new[b]], r.inv_freq, 1.0, inter).float()
        want.append(b, start[b], kr, v[b, :new[b]].cpu())
    # rotated values are off by 1e-6 (see test_rope; |x| <= 5), so scales by
    # 1e-6 / 127 and codes by one where x / scale lies near a half
    assert torch.equal(c.v_codes.cpu(), want.codes["v"])
    ok = ~torch.isnan(want.scales["k"])
    assert ((c.k_scales.cpu() - want.scales["k"]).abs()[ok] <= 1e-6 / 127 + 2 ** -23).all()
    off = (c.k_codes.cpu().int() - want.codes["k"].int()).abs()
    assert off.max() <= 1
    assert (off > 0).float().mean() < 1e-3  # 127 * 1e-6 / (amax > 1) of a unit step, twice


def test_append_skips_unmapped_blocks_and_tails():
    c, _ = filled(21, [64, 64], 1, 64, 16, unmapped=[(0, 1), (1, 3)])
    k, v = rand(22, 2, 64, 1, 64), rand(23, 2, 64, 1, 64)
    want = ref.Cache(c)
    kvq.b8_append(c, k, v, ints([0, 0]))
    for b in range(2):
        want.append(b, 0, k[b].cpu(), v[b].cpu())
    assert torch.equal(c.k_codes.cpu(), want.codes["k"])
    assert torch.equal(c.v_codes.cpu(), want.codes["v"])
    # past the table's columns and at the far end of int32: nothing is stored
    kvq.b8_append(c, k, v, ints([64, 2 ** 31 - 2]))
    assert torch.equal(c.k_codes.cpu(), want.codes["k"])
    gk, _ = kvq.b8_gather(c, ints([16, 2 ** 31 - 2]), ints([32, 2 ** 31 - 1]), 16, F32)
    assert not gk.any()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim,block,t_new", [(64, 16, 40), (256, 256, 300)])
@pytest.mark.parametrize("bad", [math.nan, -math.nan, math.inf, -math.inf])
def test_append_of_what_is_not_finite(dtype, dim, block, t_new, bad):
    """One element of one head: its block becomes NaN, the others stay as they are,
    later tokens of the block do not bring it back, and a new start does."""
    c, d = (kvq.B8Cache.contiguous(1, 2, 600, dim, block) for _ in "cd")
    k, v = rand(191, 1, t_new, 2, dim, dtype=dtype), rand(192, 1, t_new, 2, dim, dtype=dtype)
    kvq.b8_append(d, k, v, ints([0]))
    at = block + 3
    for which in "kv":
        x = {"k": k, "v": v}
        x[which] = x[which].clone()
        x[which][0, at, 1, dim - 5] = bad
        kvq.b8_append(c, x["k"], x["v"], ints([0]))
        for w, got, want in (("k", c.k_scales, d.k_scales), ("v", c.v_scales, d.v_scales)):
            want = want.clone()
            if w == which:
                want[1, 1] = math.nan
            assert torch.equal(got.isnan(), want.isnan())
            assert torch.equal(got.nan_to_num(), want.nan_to_num())
        one = torch.ones((1, 1, 2, dim), dtype=dtype, device="cuda")
        kvq.b8_append(c, one, one, ints([block + 8]))
        assert (c.k_scales if which == "k" else c.v_scales)[1, 1].isnan()
        val = kvq.b8_gather(c, ints([0]), ints([t_new]), t_new, F32)[which == "v"]
        assert val[0, block:2 * block, 1].isnan().all() and val.isnan().sum() == dim * min(
            block, t_new - block)
    kvq.b8_append(c, k, v, ints([0]))
    assert torch.equal(c.k_scales, d.k_scales) and torch.equal(c.v_scales, d.v_scales)
    assert torch.equal(c.k_codes, d.k_codes) and torch.equal(c.v_codes, d.v_codes)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gather_into_16_byte_alignment(dtype):
    c, _ = filled(61, [50, 70], 2, 128, 32)
    first, ends = ints([3, 0]), ints([50, 66])
    want = kvq.b8_gather(c, first, ends, 67, dtype)
    size, off = want[0].numel(), 16 // dtype.itemsize
    got = [torch.full((size + 2 * off,), -7.0, dtype=dtype, device="cuda") for _ in "kv"]
    views = [x[off:off + size].view(want[0].shape) for x in got]
    kvq.b8_gather(c, first, ends, 67, dtype, k_out=views[0], v_out=views[1])
    for w, v, x in zip(want, views, got):
        assert torch.equal(w, v) and (x[:off] == -7).all() and (x[-off:] == -7).all()


# ------------------------------------------------------------------ attention
def tolerance(dtype, dim, tokens, a, want, vmax):
    """Scores: q keeps 22 bits (bf16: all), each of the dim / 16 (twice that for
    hi + lo) accumulations rounds or truncates at 2^-22 of at most a, the scaling
    and the difference with the maximum at 2^-23 of it.  exp2 and the
    probability's product: 2^-20.  Sums over tokens / 16 steps, a warp's share of
    them, at 2^-23 each.  bf16: the probability is rounded to fp16 (2^-11), the
    result to bf16."""
    s = a * 2.0 ** -22 * (2 + dim / 16 * (1 if dtype == BF16 else 2)) + 2.0 ** -20
    steps = tokens / 16 * 2.0 ** -23 + 16 * 2.0 ** -23
    rel = 2 * s + steps + (2.0 ** -11 if dtype == BF16 else 0)
    out = rel[..., None] * vmax
    if dtype == BF16:
        out = out + want.abs() * torch.finfo(BF16).eps / 2
    return out, s + steps


def check_attention(c, q, lens, cu, max_len, dtype, scale, **kw):
    out, lse = kvq.b8_attn(c, q, ints(lens), max_len, scale,
                           cu_q=None if cu is None else ints(cu),
                           max_q=None if cu is None else max(np.diff(cu).max(), 1),
                           return_lse=True, **kw)
    r = ref.Cache(c)
    at = list(range(len(lens) + 1)) if cu is None else cu
    real = [min(max(n, 0), max_len) for n in lens]
    want, wlse, a = ref.attention(r, q, real, at, scale)
    scales = r.scales["v"][r.table[(r.table >= 0) & (r.table < r.nb)]]
    vmax = 127 * (scales.nan_to_num(0).max().item() if scales.numel() else 0)
    tol, ltol = tolerance(dtype, c.head_dim, max(real), a, want, vmax)
    err = (out.double().cpu() - want).abs()
    assert (err <= tol).all(), (err - tol).max()
    fin = torch.isfinite(wlse)
    got = lse.double().cpu()
    assert torch.equal(fin, torch.isfinite(got)) and (got[~fin] == -math.inf).all()
    assert ((got - wlse).abs()[fin] <= ltol[fin] + wlse.abs()[fin] * 2 ** -22).all()
    return out, lse, r, real, at, a


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 3, 8, 16])
def test_decode(dtype, dim, group):
    lens = [0, 1, 15, 16, 17, 127, 128, 129, 300, 1000]
    c, _ = filled(31 + dim, lens, 2, dim, 16 if group < 8 else 32,
                  unmapped=[(8, 2), (9, 0), (9, 5)])
    q = rand(32, len(lens), 2 * group, dim, dtype=dtype)
    check_attention(c, q, lens, None, 1000, dtype, dim ** -0.5)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("block", [16, 64, 256])
@pytest.mark.parametrize("longest,clamp", [(9001, 5000), (20001, 17000)])
def test_decode_in_splits(dtype, block, longest, clamp):
    """Long enough for several ranges, joined in a cluster or by a second kernel;
    lengths are clamped to max_seq_len, and a sequence whose blocks are all
    unmapped attends to nothing."""
    lens = [longest, 4096, 33, 500]
    c, _ = filled(41, lens, 1, 128, block, unmapped=[(3, i) for i in range((500 - 1) // block + 1)])
    q = rand(42, 4, 4, 128, dtype=dtype)
    assert (kvq.b8_attn_workspace(c, 4, 4, longest) > 0) == (longest > 16384)
    check_attention(c, q, lens, None, longest, dtype, 0.05)
    check_attention(c, q, [longest, 4096, -7, 500], None, clamp, dtype, 0.05)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim,group,nq,lens", [
    (64, 4, [1, 2, 3], [1, 100, 2]), (128, 1, [5, 0, 70], [70, 10, 70]),
    (128, 5, [33, 17, 64], [33, 500, 40]), (128, 4, [130, 200], [1000, 200]),
    (256, 8, [9, 40], [2000, 40]), (256, 2, [129, 65], [260, 64]), (128, 16, [3, 9], [300, 8]),
    (64, 2, [300, 140], [700, 141])])
def test_causal_prompts(dtype, dim, group, nq, lens):
    """Ragged queries; more queries than tokens leave the first ones empty."""
    c, _ = filled(51 + dim, lens, 2, dim, 32, unmapped=[(0, 1)] if lens[0] > 40 else [])
    x = rand(52, sum(nq) + 3, 2 * group + 4, dim, dtype=dtype)
    cu = [0] + np.cumsum(nq).tolist()
    q = x[:sum(nq), 2:2 + 2 * group]
    out, lse, r, real, at, a = check_attention(c, q, lens, cu, max(lens), dtype, dim ** -0.5)
    # rows of no sequence stay as they were, in padded buffers too
    big = torch.full((sum(nq) + 3, 2 * group, dim), 7.0, dtype=dtype, device="cuda")
    blse = torch.full(big.shape[:2], 7.0, device="cuda")
    kvq.b8_attn(c, x[:, 2:2 + 2 * group], ints(lens), max(lens), dim ** -0.5, cu_q=ints(cu),
                max_q=max(nq), out=big, lse=blse)
    assert torch.equal(big[:sum(nq)], out) and (big[sum(nq):] == 7).all()
    assert torch.equal(blse[:sum(nq)], lse) and (blse[sum(nq):] == 7).all()
    # the weights of the same queries
    m0 = torch.rand((len(lens), 2, max(lens) + 5), generator=torch.Generator().manual_seed(1))
    m = m0.cuda()
    kvq.b8_attn_mass(c, q, lse, ints(lens), max(lens), dim ** -0.5, m, cu_q=ints(cu),
                     max_q=max(nq))
    check_mass(m, m0, r, q, lse, real, at, dim ** -0.5, a, dtype)


def check_mass(m, m0, r, q, lse, real, at, scale, a, dtype):
    want = ref.mass(r, q, lse, real, at, scale, m0)
    # each weight: its score (see tolerance) and lse in log2 units (2^-22 of
    # them), then sums over rows
    fin = lse[torch.isfinite(lse)]
    big = fin.abs().max().item() if fin.numel() else 0.0
    dim = q.shape[2]
    s = a.max().item() * 2.0 ** -22 * (2 + dim / 16 * 2) + 2.0 ** -20 + 2 * (big + 1) * 2.0 ** -22
    rows = max(np.diff(at)) * q.shape[1]
    tol = (want - m0.double()) * (2 * s + rows * 2.0 ** -24) + want.abs() * 2.0 ** -23
    err = (m.double().cpu() - want).abs()
    assert (err <= tol).all(), (err - tol).max()
    for b, n in enumerate(real):  # behind the length: as it was
        assert torch.equal(m[b, :, n:].cpu(), m0[b, :, n:])


@pytest.mark.parametrize("batch,hkv,group,most_q,longest", [
    (6, 8, 4, 220, 700),    # more units than SMs: whole ones, and cut ones at the end
    (600, 1, 16, 8, 90)])   # more sequences than a CTA ranks
def test_prompts_of_many_units(batch, hkv, group, most_q, longest):
    g = np.random.default_rng(batch)
    lens = g.integers(0, longest + 1, batch).tolist()
    nq = np.minimum(g.integers(0, most_q + 1, batch), 10 + np.array(lens)).tolist()
    lens[0], nq[0] = longest, most_q
    c, _ = filled(55, lens, hkv, 64, 16)
    q = rand(56, sum(nq), hkv * group, 64, dtype=BF16)
    check_attention(c, q, lens, [0] + np.cumsum(nq).tolist(), longest, BF16, 0.125)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim,group", [(64, 1), (128, 4), (128, 16), (256, 5)])
def test_mass_of_decode_steps(dtype, dim, group):
    lens = [0, 1, 16, 31, 257, 5000]
    c, _ = filled(61, lens, 2, dim, 16, unmapped=[(5, 3), (4, 0)])
    q = rand(62, len(lens), 2 * group, dim, dtype=dtype)
    out, lse, r, real, at, a = check_attention(c, q, lens, None, 5000, dtype, dim ** -0.5)
    m0 = torch.rand((len(lens), 2, 5000), generator=torch.Generator().manual_seed(2))
    m = m0.cuda()
    kvq.b8_attn_mass(c, q, lse, ints(lens), 5000, dim ** -0.5, m)
    check_mass(m, m0, r, q, lse, real, at, dim ** -0.5, a, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_wide_ranges_of_values(dtype):
    """Block scales from 2^-60 to 2^60, zero scales, query rows from 2^-30 to
    2^30, and scores of some hundreds: nothing overflows on the way."""
    c, _ = filled(71, [400, 400], 1, 128, 16)
    nb = c.num_blocks
    e = torch.linspace(-60, 60, nb, device="cuda")[:, None]
    c.v_scales.copy_(torch.exp2(e))
    c.v_scales[3] = 0
    c.v_codes[3] = 0
    q = rand(72, 2, 4, 128)
    q[0, 0] *= 2.0 ** -30
    q[0, 1] *= 2.0 ** 9
    q[1, 2] = 0
    c.k_scales.nan_to_num_(1.0)
    check_attention(c, q.to(dtype), [400, 390], None, 400, dtype, 0.1)
    q[1, 3] *= 2.0 ** 30
    c.k_scales.mul_(2.0 ** -30)
    check_attention(c, q.to(dtype), [400, 390], None, 400, dtype, 0.1)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("nq,span", [(1, 10), (1, 30), (1, 60), (3, 10), (3, 30), (3, 60), (80, 10),
                                     (80, 30), (80, 45)])
@pytest.mark.parametrize("lean", [0.0, 0.5, 1.0, 2.0])
@pytest.mark.parametrize("zeros", [False, True])
def test_blocks_of_far_scales(dtype, nq, span, lean, zeros):
    """V block scales from 2^-span to 2^span in any order.  Each token's score is
    -lean * log(scale): at 2 the weight lies on the smallest scales and the largest
    ones, seen or masked, add nothing.  The error is counted in what each row's own
    tokens weigh, not in the cache's largest scale."""
    dim, block, n = 128, 16, 6000 + 4 * nq  # several tiles a warp
    c, _ = filled(171, [n], 1, dim, block)
    cols = c.block_table.shape[1]
    g = torch.Generator().manual_seed(172)
    e = torch.linspace(-span, span, cols)[torch.randperm(cols, generator=g)]
    pages = c.block_table[0].long().cpu()
    ks, vs, kc = (x.cpu().clone() for x in (c.k_scales, c.v_scales, c.k_codes))
    ks[pages] = 0.5
    vs[pages] = torch.exp2(e + torch.rand(cols, generator=g))[:, None]
    kc[pages] = (kc[pages].float() / 6).round().to(torch.int8)
    kc[pages, :, :, 0] = (-lean * math.log(2) * e).round().to(torch.int8)[:, None, None]
    if zeros:  # most of the weight on a block of zeros
        vs[pages[3]] = 0
        c.v_codes[pages[3].item()] = 0
        kc[pages[3], :, :, 0] = kc[pages, 0, 0, 0].max() + 8
    c.k_scales.copy_(ks), c.v_scales.copy_(vs), c.k_codes.copy_(kc)
    q = rand(173, nq, 4, dim) / 50
    q[..., 0] = 2.0
    q = q.to(dtype)
    cu = [0, nq]
    out, lse = kvq.b8_attn(c, q, ints([n]), n, 1.0, cu_q=ints(cu), max_q=nq, return_lse=True)
    r = ref.Cache(c)
    want, wlse, a = ref.attention(r, q, [n], cu, 1.0)
    k, _ = r.values("k", 0, n)
    v, _ = r.values("v", 0, n)
    see = torch.arange(n)[None] <= n - nq + torch.arange(nq)[:, None]
    s = torch.einsum("qhd,td->qht", q.double().cpu(), k[0]).masked_fill(~see[:, None], -math.inf)
    p = torch.exp(s - wlse[..., None])
    scale_of = r.scales["v"][r.table[0]].double()[:, 0].repeat_interleave(block)[:n]
    # P * v_scale: fp16's half step of itself, or of its subnormals, 2^-25, in
    # units where the row's largest is 2^5 at least, or 2^3 with many rows, where a
    # scale up to 4 times its own may set them (see `tolerance` for the rest).
    # Weights below 2^-112 of the row's largest leave fp32's range on the way.
    gone = torch.where(p < p.amax(-1, keepdim=True) * 2.0 ** -112, p, 0.0)
    tol, ltol = tolerance(dtype, dim, n, a, want * 0, torch.tensor(1.0))
    tol = (tol * (p @ v[0].abs())
           + 2.0 ** (-30 if nq < 48 else -28) * (p * scale_of).amax(-1, keepdim=True) * 127 * n
           + gone @ v[0].abs() + want.abs() * (2.0 ** -8 if dtype == BF16 else 2.0 ** -24))
    err = (out.double().cpu() - want).abs()
    assert (err <= tol).all(), (err / tol).max()
    assert ((lse.double().cpu() - wlse).abs() <= ltol + wlse.abs() * 2.0 ** -22).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("nq", [1, 40, 140])
def test_scales_as_far_as_they_go(dtype, nq):
    """Scales of 2^-107 and 2^100, weights that lean 2^-240 the other way: what
    fp32 cannot hold counts as nothing, and nothing becomes NaN."""
    n, block = 4000, 16
    c, _ = filled(174, [n], 1, 64, block)
    c.k_codes[..., 0] = 127
    big = torch.arange(c.num_blocks, device="cuda") % 2 == 1
    for hi, lo in ((100, -107), (61, -60), (50, -20)):
        c.v_scales[:] = torch.where(big, 2.0 ** hi, 2.0 ** lo)[:, None]
        for lean in (-1.2, -1.0, -0.9, 0.9, 1.0):
            # q . k * scale: 127 * k_scale, natural units
            c.k_scales[:] = torch.where(big, lean, 0.0)[:, None] * (hi - lo) * math.log(2) / 127
            c.k_scales.abs_()
            q = torch.zeros((nq, 1, 64), device="cuda", dtype=dtype)
            q[..., 0] = math.copysign(1.0, lean)
            out, lse = kvq.b8_attn(c, q, ints([n]), n, 1.0, cu_q=ints([0, nq]), max_q=nq,
                                   return_lse=True)
            assert torch.isfinite(out).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("nq", [1, 45, 140])
def test_scales_near_the_ends_of_fp32(dtype, nq):
    """One scale for all blocks, up to what the header allows: exact; past that, no
    finite number that is wrong."""
    n = 300
    c, _ = filled(179, [n], 1, 64, 16)
    q = rand(180, nq, 2, 64, dtype=dtype)
    for e in (-107, -60, 0, 60, 100, 104):
        c.v_scales.fill_(2.0 ** e)
        out, *_ = check_attention(c, q, [n], [0, nq], n, dtype, 0.05)
        assert out.any()
    c.v_scales.fill_(2.0 ** 110)
    out, lse = kvq.b8_attn(c, q, ints([n]), n, 0.05, cu_q=ints([0, nq]), max_q=nq, return_lse=True)
    r = ref.Cache(c)
    want, wlse, _ = ref.attention(r, q, [n], [0, nq], 0.05)
    good = torch.isfinite(out).cpu()
    assert ((out.double().cpu() - want).abs()[good] <= 2.0 ** 117 * 2.0 ** -7).all()
    good = torch.isfinite(lse).cpu()
    assert ((lse.double().cpu() - wlse).abs()[good] < 1e-4).all()
    assert not (lse == -math.inf).any()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("block,nq,group,last", [(16, 3, 1, 1), (16, 20, 2, 7), (64, 70, 4, 5),
                                                 (16, 140, 1, 16), (32, 40, 8, 30)])
@pytest.mark.parametrize("which", ["k", "v"])
def test_a_bad_block_spoils_the_rows_that_see_it_only(dtype, block, nq, group, last, which):
    """The last block, of `last` tokens, holds NaN; the first queries end before it."""
    n = 10 * block + last
    c, _ = filled(195, [n], 1, 128, block)
    q = rand(196, nq, group, 128, dtype=dtype)
    kw = dict(cu_q=ints([0, nq]), max_q=nq)
    m = [torch.zeros((1, 1, n), device="cuda") for _ in range(2)]
    want, wlse = kvq.b8_attn(c, q, ints([n]), n, 0.1, return_lse=True, **kw)
    kvq.b8_attn_mass(c, q, wlse, ints([n]), n, 0.1, m[0], **kw)
    (c.k_scales if which == "k" else c.v_scales)[c.block_table[0, -1].long()] = math.nan
    out, lse = kvq.b8_attn(c, q, ints([n]), n, 0.1, return_lse=True, **kw)
    kvq.b8_attn_mass(c, q, wlse, ints([n]), n, 0.1, m[1], **kw)
    sees = nq - last
    assert torch.equal(out[:sees], want[:sees]) and torch.equal(lse[:sees], wlse[:sees])
    assert torch.isnan(out[sees:]).all()
    assert torch.equal(m[0][..., :n - last], m[1][..., :n - last])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("scale", [0.0, -0.125])
def test_other_scales(dtype, scale):
    c, _ = filled(73, [300, 40], 1, 64, 32)
    for nq in (1, 40):
        q = rand(74, 2 * nq, 4, 64, dtype=dtype)
        check_attention(c, q, [300, 40], [0, nq, 2 * nq], 300, dtype, scale)


def test_nothing_cached_and_one_kv_head_for_many():
    """No token at all, by every kernel; 144 query heads on one kv head."""
    c, _ = filled(75, [64, 64], 1, 128, 64)
    for dtype, nq, hq in ((BF16, 1, 4), (F32, 1, 16), (F32, 9, 4), (BF16, 70, 2)):
        q = rand(76, 2 * nq, hq, 128, dtype=dtype)
        for lens, most in (([0, 0], 64), ([64, 64], 0)):
            out, lse = kvq.b8_attn(c, q, ints(lens), most, 0.1, cu_q=ints([0, nq, 2 * nq]), max_q=nq,
                                   return_lse=True)
            assert not out.any() and (lse == -math.inf).all()
    for dtype in (BF16, F32):
        check_attention(c, rand(77, 2, 144, 128, dtype=dtype), [64, 33], None, 64, dtype, 0.08)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("nq", [1, 3, 80])
def test_a_bad_query_spoils_its_own_row_only(dtype, nq):
    c, _ = filled(78, [500], 1, 128, 16)
    q = rand(79, nq, 2, 128, dtype=dtype)
    kw = dict(cu_q=ints([0, nq]), max_q=nq, return_lse=True)
    want, wlse = kvq.b8_attn(c, q, ints([500]), 500, 0.1, **kw)
    for v in (math.nan, math.inf):
        bad = q.clone()
        bad[0, 1, 7] = v
        out, lse = kvq.b8_attn(c, bad, ints([500]), 500, 0.1, **kw)
        assert torch.isnan(out[0, 1]).all() and torch.isnan(lse[0, 1])
        ok = torch.ones((nq, 2), dtype=torch.bool, device="cuda")
        ok[0, 1] = False
        assert torch.equal(out[ok], want[ok]) and torch.equal(lse[ok], wlse[ok])


def test_two_calls_at_once():
    """Prompts, decodes and weights on two streams at the same time."""
    c, _ = filled(83, [3000, 2500], 2, 128, 64)
    q = rand(84, 600, 8, 128, dtype=BF16)
    p = dict(cu_q=ints([0, 300, 600]), max_q=300, return_lse=True)
    lens, d = ints([3000, 2500]), q[:2].contiguous()
    want, wlse = kvq.b8_attn(c, q, lens, 3000, 0.08, **p)
    dec, dlse = kvq.b8_attn(c, d, lens, 3000, 0.08, return_lse=True)
    m0 = torch.zeros((2, 2, 3000), device="cuda")
    kvq.b8_attn_mass(c, d, dlse, lens, 3000, 0.08, m0)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for i in range(6):
        for st in streams:
            a = kvq.b8_attn(c, q, lens, 3000, 0.08, stream=st, **p)[0]
            b, l = kvq.b8_attn(c, d, lens, 3000, 0.08, stream=st, return_lse=True)
            with torch.cuda.stream(st):
                m = torch.zeros((2, 2, 3000), device="cuda")
            kvq.b8_attn_mass(c, d, l, lens, 3000, 0.08, m, stream=st)
            got.append((a, b, m))
    torch.cuda.synchronize()
    for a, b, m in got:
        assert torch.equal(a, want) and torch.equal(b, dec) and torch.equal(m, m0)


def test_wait_timeout_is_reported_and_recovers():
    """A wait of the many-row kernel that gives up at once leaves NaN and a flag;
    the next call with the default limit is exact again."""
    c, _ = filled(85, [4000], 2, 128, 64)
    q = rand(86, 512, 8, 128, dtype=BF16)
    run = lambda: kvq.b8_attn(c, q, ints([4000]), 4000, 0.08, cu_q=ints([0, 512]), max_q=512)
    want = run()
    assert kvq.device_errors() == 0
    kvq.set_wait_limit(0)
    try:
        got = run()
        flags = kvq.device_errors()
    finally:
        kvq.set_wait_limit(-1)
    assert flags & kvq.KVQ_DEVERR_WAIT_TIMEOUT
    assert torch.isnan(got).any()
    again = run()
    assert kvq.device_errors() == 0
    assert torch.equal(again, want)


def test_waits_that_run_out_at_any_place():
    """Limits that let a wait of any role run out, early, late or never: a row is
    NaN or exact, NaN comes with the flag, and calls beside and after it, which
    may take over its multiprocessors' memory, are exact."""
    c, _ = filled(87, [2500, 700], 2, 128, 64)
    q = rand(88, 300, 8, 128, dtype=BF16)
    args = (c, q, ints([2500, 700]), 2500, 0.08)
    kw = dict(cu_q=ints([0, 200, 300]), max_q=200, return_lse=True)
    want, wlse = kvq.b8_attn(*args, **kw)
    assert kvq.device_errors() == 0
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for polls in list(range(12)) + [16, 24, 40, 80, 200]:
        kvq.set_wait_limit(polls)
        try:
            got = [kvq.b8_attn(*args, **kw) for _ in range(3)]
        finally:
            kvq.set_wait_limit(-1)
        after = [kvq.b8_attn(*args, **kw), kvq.b8_attn(*args, stream=side, **kw)]
        flags = kvq.device_errors()  # synchronises
        bad = False
        for out, lse in got:
            nan = torch.isnan(lse)
            assert torch.equal(out[~nan], want[~nan]) and torch.equal(lse[~nan], wlse[~nan])
            assert torch.isnan(out[nan]).all()
            bad |= bool(nan.any())
        assert not bad or flags == kvq.KVQ_DEVERR_WAIT_TIMEOUT
        for out, lse in after:
            assert torch.equal(out, want) and torch.equal(lse, wlse)


def test_bad_query_ranges_have_no_queries():
    c, _ = filled(81, [50, 50, 50], 1, 64, 16)
    q = rand(82, 12, 2, 64)
    out = torch.full_like(q, 5.0)
    for cu in ([0, 4, 13, 13], [0, 4, 3, 3], [-1, -1, 12, 12], [0, 9, 12, 12]):
        lse = torch.full((12, 2), 5.0, device="cuda")
        kvq.b8_attn(c, q, ints([50] * 3), 50, 0.1, cu_q=ints(cu), max_q=8, out=out, lse=lse)
        m = torch.zeros((3, 1, 50), device="cuda")
        kvq.b8_attn_mass(c, q, torch.zeros((12, 2), device="cuda"), ints([50] * 3), 50, 0.1, m,
                         cu_q=ints(cu), max_q=8)
        for b in range(3):
            n = cu[b + 1] - cu[b]
            ok = cu[b] >= 0 and 0 < n <= 8 and cu[b + 1] <= 12
            assert bool(m[b].any()) == ok
            if ok:
                assert not (out[cu[b]:cu[b + 1]] == 5).any()
                out[cu[b]:cu[b + 1]] = 5.0
        assert (out == 5).all()


# ------------------------------------------------------------------ eviction
@pytest.mark.parametrize("dim,block,to_block", [(64, 16, 16), (128, 32, 64), (256, 256, 256),
                                                (128, 128, 16)])
@pytest.mark.parametrize("keep,recent,sinks", [(1, 0, 0), (40, 8, 4), (64, 0, 0), (50, 30, 20),
                                               (300, 100, 3)])
def test_evict(dim, block, to_block, keep, recent, sinks):
    lens = [0, 1, 39, 40, 41, 299, 301, 700]
    c, _ = filled(91 + dim, lens, 2, dim, block, unmapped=[(7, 0)])
    batch, n = len(lens), max(lens)
    g = torch.Generator().manual_seed(keep)
    m = torch.exp(2 * torch.randn((batch, 2, n + 3), generator=g))
    m[:, 0] = (m[:, 0] * 2).round() / 2  # many ties, many zeros
    m[7, 1, ::5] = 0.0
    m[7, 1, 2::5] = -0.0
    m[6, 1, 17] = math.inf
    m[6, 1, 18] = math.nan
    m[5, 1, 20] = -1.0
    cols = (keep + to_block - 1) // to_block
    into, _ = filled(92, [cols * to_block] * batch, 2, dim, to_block)
    want, dst = ref.Cache(c), ref.Cache(into)
    ln, kept, mo = kvq.b8_evict(c, into, m.cuda(), ints(lens), n, keep, recent=recent, sinks=sinks)
    assert ln.tolist() == [min(x, keep) for x in lens]
    for b in range(batch):
        ids = want.evict(dst, b, lens[b], m[b], keep, recent, sinks)
        for h in range(2):
            k = len(ids[h])
            assert kept[b, h, :k].tolist() == ids[h]
            assert (kept[b, h, k:] == -1).all() and (mo[b, h, k:] == 0).all()
            assert torch.equal(mo[b, h, :k].cpu().view(torch.int32),
                               m[b, h, ids[h]].view(torch.int32))
    # the fp32 operations are pinned: bit-exact, rows behind the last untouched
    for w, codes, scales in (("k", into.k_codes, into.k_scales), ("v", into.v_codes, into.v_scales)):
        assert torch.equal(codes.cpu(), dst.codes[w])
        assert torch.equal(scales.cpu().view(torch.int32), dst.scales[w].view(torch.int32))


def test_evict_long_and_equal_weights():
    """More tokens than one pass of the threads, all weights equal: the lowest
    indices stay."""
    n, keep = 70000, 5000
    table = torch.arange(n // 16 + 1 + (keep + 15) // 16, dtype=torch.int32)
    c = kvq.B8Cache(table.numel(), 1, 16, 64, table[None, :n // 16 + 1].cuda())
    into = c.with_block_table(table[None, n // 16 + 1:].cuda())
    c.k_codes.random_(-127, 128)
    c.k_scales.fill_(0.5)
    m = torch.full((1, 1, n), 0.25, device="cuda")
    _, kept, _ = kvq.b8_evict(c, into, m, ints([n]), n, keep, recent=100, sinks=7)
    want = list(range(keep - 100)) + list(range(n - 100, n))
    assert kept[0, 0].tolist() == want
    wide = torch.empty((1, 1, keep + 50), device="cuda")
    kvq.b8_evict(c, into, m, ints([n]), n, keep, mass_out=wide)
    assert (wide[..., :keep] == 0.25).all() and (wide[..., keep:] == 0).all()


@pytest.mark.parametrize("dim,block,to_block", [(64, 16, 32), (128, 32, 16), (256, 256, 256)])
def test_evict_carries_nan_along(dim, block, to_block):
    """A block of a NaN scale: where one of its tokens is kept, the block that it comes
    to is NaN; where none is, nothing of it is left."""
    n, keep = 3 * block, 2 * block
    c, _ = filled(193, [n], 2, dim, block)
    into, _ = filled(194, [keep], 2, dim, to_block)
    page = c.block_table[0].long()
    c.k_scales[page[1], 0] = math.nan
    c.v_scales[page[2], 1] = math.nan
    m = torch.ones((1, 2, n), device="cuda")
    m[0, 0, block + 1:2 * block] = 0.0  # one token of K's block stays
    m[0, 1, 2 * block:] = 0.0           # none of V's
    _, kept, _ = kvq.b8_evict(c, into, m, ints([n]), n, keep)
    k, v = kvq.b8_gather(into, ints([0]), ints([keep]), keep, F32)
    at = kept[0, 0].tolist().index(block)
    one = torch.zeros(keep, dtype=torch.bool, device="cuda")
    one[at // to_block * to_block:(at // to_block + 1) * to_block] = True
    assert torch.equal(k[0, :, 0].isnan().all(-1), one) and torch.equal(k[0, :, 0].isnan().any(-1), one)
    assert not k[:, :, 1].isnan().any() and not v.isnan().any()


@pytest.mark.parametrize("keep", [64, 40])
def test_evicted_tokens_without_a_block_become_zeros(keep):
    """Left out by attention before, rows of zeros of score 0 afterwards, whether
    tokens were dropped or not."""
    c, _ = filled(94, [64], 2, 64, 16, unmapped=[(0, 1)])
    into, _ = filled(95, [64], 2, 64, 16)
    q = rand(96, 1, 4, 64)
    before = kvq.b8_attn(c, q, ints([64]), 64, 0.1, return_lse=True)[1]
    m = torch.zeros((1, 2, 64), device="cuda")
    m[:, :, 16:32] = 1.0  # the heaviest are those without a block
    ln, kept, _ = kvq.b8_evict(c, into, m, ints([64]), 64, keep)
    assert ln.tolist() == [keep] and (kept[0, :, :keep] == torch.arange(keep, device="cuda")).all()
    k, v = kvq.b8_gather(into, ints([0]), ints([keep]), keep, F32)
    old_k, _ = kvq.b8_gather(c, ints([0]), ints([64]), 64, F32)
    assert not k[:, 16:32].any() and not v[:, 16:32].any() and k[:, :16].any()
    _, after, _, _, _, _ = check_attention(into, q, [keep], None, keep, F32, 0.1)
    if keep == 64:
        # 16 terms of exp(0) more.  Every block holds a code of 127 or -127, so its
        # codes stay and its scale is rounded twice, 2^-24 each: scores below 32 and
        # their sums are off by 2^-17 at most.
        assert torch.allclose(k[:, 32:], old_k[:, 32:], rtol=2 ** -22)
        want = torch.log(torch.exp(before.double()) + 16)
        assert ((after.double() - want).abs() < 2 ** -16).all()


def far_table(first, cols, bs, n):
    """A table of `cols` columns whose blocks are mapped from column `first` on."""
    t = torch.full((1, cols), -1, dtype=torch.int32, device="cuda")
    t[0, first:first + n] = torch.arange(n, dtype=torch.int32, device="cuda")
    return t


def near_and_far(dim, hkv, tail):
    """The same last tokens at the end of a short table and of one of almost 2^31
    tokens, the others unmapped: (cache, length) twice."""
    bs, n = 256, 6
    g = torch.Generator().manual_seed(175)
    codes = [torch.randint(-127, 128, (n, hkv, bs, dim), generator=g, dtype=torch.int8).cuda()
             for _ in "kv"]
    scales = [torch.rand((n, hkv), generator=g).cuda() / 64 for _ in "kv"]
    cols = (2 ** 31 - 4096) // bs - 1
    far = kvq.B8Cache.wrap(codes[0], scales[0], codes[1], scales[1], far_table(cols - n, cols, bs, n))
    near = far.with_block_table(far_table(0, n, bs, n))
    return (near, n * bs - tail), (far, cols * bs - tail)


@pytest.mark.parametrize("dtype,hkv,hq", [(BF16, 1, 1), (F32, 1, 16), (BF16, 4, 4)])
def test_decode_at_the_end_of_the_longest_table(dtype, hkv, hq):
    q = rand(176, 1, hq, 64, dtype=dtype)
    got = [kvq.b8_attn(c, q, ints([n]), n, 0.1, return_lse=True)
           for c, n in near_and_far(64, hkv, 37)]
    # The same tokens in other splits.  Each side: 1499 / 16 sums at 2^-23, exp2 and
    # scores below 16 at 2^-19, and for bf16 11 bits of P, of at most 2 (the largest
    # value), then one rounding.
    tol = 2 * 2 * (94 * 2.0 ** -23 + 2.0 ** -19 + (2.0 ** -11 if dtype == BF16 else 0.0))
    if dtype == BF16:
        tol = tol + 2 * 2.0 ** -8 * got[0][0].abs()
    assert got[0][0].any()
    assert ((got[0][0] - got[1][0]).abs() <= tol).all()
    assert ((got[0][1] - got[1][1]).abs() <= 2.0 ** -15).all()


def test_prompt_at_the_end_of_the_longest_table():
    q = rand(178, 130, 1, 64, dtype=BF16)
    got = [kvq.b8_attn(c, q, ints([n]), n, 0.1, cu_q=ints([0, 130]), max_q=130, return_lse=True)
           for c, n in near_and_far(64, 1, 37)]
    # the same tokens in other pieces: see the decode above, 24 tiles' sums a piece
    tol = 4 * (94 * 2.0 ** -23 + 2.0 ** -19 + 2.0 ** -11) + 2 * 2.0 ** -8 * got[0][0].abs()
    assert got[0][0].any()
    assert ((got[0][0] - got[1][0]).abs() <= tol).all()
    assert ((got[0][1] - got[1][1]).abs() <= 2.0 ** -15).all()


@pytest.mark.parametrize("dtype,nq", [(BF16, 1), (F32, 1), (BF16, 20), (F32, 20)])
def test_mass_at_the_end_of_the_longest_table(dtype, nq):
    q = rand(177, nq, 2, 64, dtype=dtype)
    kw = dict(cu_q=ints([0, nq]), max_q=nq)
    got, lse = [], None
    for c, n in near_and_far(64, 1, 37):
        m = torch.zeros((1, 1, n), device="cuda")
        if lse is None:
            lse = kvq.b8_attn(c, q, ints([n]), n, 0.1, return_lse=True, **kw)[1]
        kvq.b8_attn_mass(c, q, lse, ints([n]), n, 0.1, m, **kw)
        got.append(m[0, 0, n - 1400:].clone())
    # a token's sum has the same order in every split
    assert got[0].all() and torch.equal(*got)


def test_evict_nothing():
    """A batch without a token, of a longest length of 0."""
    c, _ = filled(95, [0, 0], 2, 64, 16)
    into, _ = filled(96, [16, 16], 2, 64, 16)
    before = into.k_codes.clone()
    ln, kept, mo = kvq.b8_evict(c, into, torch.zeros((2, 2, 0), device="cuda"), ints([0, 0]), 0, 9)
    assert ln.tolist() == [0, 0] and (kept == -1).all() and (mo == 0).all()
    assert torch.equal(before, into.k_codes)


def test_append_of_a_batch_padded_without_end():
    """The padded length sets no cost and passes no range: only 3 tokens are there."""
    k, v = rand(97, 1, 1, 2, 64, dtype=BF16), rand(98, 1, 1, 2, 64, dtype=BF16)
    a, b = (kvq.B8Cache.contiguous(1, 2, 64, 64, 32) for _ in "ab")
    most = (1 << 31) - 1
    kvq.b8_append(a, k.expand(1, most, 2, 64), v.expand(1, most, 2, 64), ints([30]),
                  new_lens=ints([3]))
    kvq.b8_append(b, k.expand(1, 3, 2, 64), v.expand(1, 3, 2, 64), ints([30]))
    assert torch.equal(a.k_codes, b.k_codes) and torch.equal(a.v_codes, b.v_codes)
    assert torch.equal(a.k_scales, b.k_scales) and torch.equal(a.v_scales, b.v_scales)
    assert (a.k_scales > 0).any()


# ------------------------------------------------------------------ as used
def test_large_planes():
    """Blocks beyond 2^32 bytes of a plane."""
    bs, hkv, dim = 256, 8, 256
    nb = (1 << 32) // (bs * hkv * dim) + 8
    table = torch.tensor([[nb - 1, 2, nb - 3]], dtype=torch.int32)
    c = kvq.B8Cache(nb, hkv, bs, dim, table.cuda())
    k, v = rand(101, 1, 700, hkv, dim, dtype=BF16), rand(102, 1, 700, hkv, dim, dtype=BF16)
    kvq.b8_append(c, k, v, ints([0]))
    small = kvq.B8Cache(3, hkv, bs, dim, ints([[0, 1, 2]]))
    kvq.b8_append(small, k, v, ints([0]))
    q = rand(103, 40, 16, dim, dtype=BF16)
    args = (q, ints([700]), 700, 1 / 16)
    kw = dict(cu_q=ints([0, 40]), max_q=40, return_lse=True)
    a, b = kvq.b8_attn(c, *args, **kw), kvq.b8_attn(small, *args, **kw)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ms = [torch.zeros((1, hkv, 700), device="cuda") for _ in "ab"]
    for x, m in zip((c, small), ms):
        kvq.b8_attn_mass(x, q, a[1], ints([700]), 700, 1 / 16, m, cu_q=ints([0, 40]), max_q=40)
    assert torch.equal(*ms)
    out = [kvq.b8_gather(x, ints([0]), ints([700]), 700) for x in (c, small)]
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
    ev = [kvq.b8_evict(c, c.with_block_table(ints([[nb - 5]])), ms[0], ints([700]), 700, 200),
          kvq.b8_evict(small, kvq.B8Cache(1, hkv, bs, dim, ints([[0]])), ms[1], ints([700]), 700,
                       200)]
    assert torch.equal(ev[0][1], ev[1][1])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_serving_path(dtype):
    """Prompt, decode steps that add up their weights, eviction, more steps with
    true positions: the whole path against attention in fp64 over the values
    the cache gives back."""
    B, hq, hkv, dim, bs = 2, 8, 2, 128, 16
    r = kvq.Rope.make(dim)
    lens = [100, 61]
    c = kvq.B8Cache(40, hkv, bs, dim, torch.randperm(40, generator=torch.Generator().manual_seed(3))
                    .int().view(2, 20).cuda())
    main, spare = c.with_block_table(c.block_table[:, :12]), c.with_block_table(
        c.block_table[:, 12:])
    k, v = rand(111, B, 100, hkv, dim, dtype=dtype), rand(112, B, 100, hkv, dim, dtype=dtype)
    kvq.b8_append(main, k, v, ints([0, 0]), new_lens=ints(lens), rope=r)
    m = torch.zeros((B, hkv, 192), device="cuda")
    true_pos = list(lens)
    cache = main
    for step in range(12):
        x = rand(120 + step, B, hq + 2 * hkv, dim, dtype=dtype)
        q, kn, vn = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        pos = ints(true_pos)
        qr, _ = kvq.rope(q, None, pos, r)
        kvq.b8_append(cache, kn[:, None], vn[:, None], ints(lens), rope=r, positions=pos[:, None])
        lens = [n + 1 for n in lens]
        true_pos = [n + 1 for n in true_pos]
        out, lse, rc, real, at, a = check_attention(cache, qr, lens, None, 192, dtype, dim ** -0.5)
        m0 = m.cpu()
        kvq.b8_attn_mass(cache, qr, lse, ints(lens), 192, dim ** -0.5, m)
        check_mass(m, m0, rc, qr, lse, real, at, dim ** -0.5, a, dtype)
        if step == 7:
            wide, before = torch.empty_like(m), m.cpu()
            want, dst = ref.Cache(cache), ref.Cache(spare)
            ln, kept, m = kvq.b8_evict(cache, spare, m, ints(lens), 192, 48, recent=16, sinks=4,
                                       mass_out=wide)
            for b in range(B):
                ids = want.evict(dst, b, lens[b], before[b], 48, 16, 4)
                assert kept[b].tolist() == ids
            assert torch.equal(spare.k_codes.cpu(), dst.codes["k"])
            assert torch.equal(spare.v_codes.cpu(), dst.codes["v"])
            lens = ln.tolist()
            assert lens == [48, 48]
            cache = spare


def test_streams_graphs_and_workspaces():
    """Two graphs that share a workspace replay in turn, a call on another stream
    with its own: the same results as an eager call; repeats are bit-identical."""
    c, _ = filled(131, [6000, 3000], 2, 128, 32)
    big = kvq.B8Cache.wrap(c.k_codes, c.k_scales, c.v_codes, c.v_scales, torch.cat(
        (c.block_table, torch.full((2, 400), -1, dtype=torch.int32, device="cuda")), 1))
    c, M = big, 18000  # a length bound that needs a workspace
    q = rand(132, 2, 8, 128, dtype=BF16)
    lens = ints([6000, 3000])
    want, wlse = kvq.b8_attn(c, q, lens, M, 0.08, return_lse=True)
    m = torch.zeros((2, 2, M), device="cuda")
    kvq.b8_attn_mass(c, q, wlse, lens, M, 0.08, m)
    assert kvq.b8_attn_workspace(c, 2, 8, M) > 0
    ws = torch.empty(kvq.b8_attn_workspace(c, 2, 8, M), dtype=torch.uint8, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    outs, graphs = [], []
    with torch.cuda.stream(st):
        for i in range(2):
            out, lse = torch.empty_like(q), torch.empty_like(wlse)
            mm = torch.zeros_like(m)
            qi = q.clone() if i == 0 else (q * 0.5)
            kvq.b8_attn(c, qi, lens, M, 0.08, out=out, lse=lse, workspace=ws)
            st.synchronize()
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr, stream=st):
                kvq.b8_attn(c, qi, lens, M, 0.08, out=out, lse=lse, workspace=ws)
                kvq.b8_attn_mass(c, qi, lse, lens, M, 0.08, mm)
            outs.append((out, lse, mm, qi))
            graphs.append(gr)
        for o in outs:
            o[0].zero_(), o[2].zero_()
        for gr in (graphs[0], graphs[1], graphs[1], graphs[0]):
            gr.replay()
    st.synchronize()
    assert torch.equal(outs[0][0], want) and torch.equal(outs[0][1], wlse)
    assert torch.equal(outs[0][2], m + m)
    half = kvq.b8_attn(c, outs[1][3], lens, M, 0.08)
    assert torch.equal(outs[1][0], half)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        o = kvq.b8_attn(c, q, lens, M, 0.08, stream=other)
        other.synchronize()
        assert torch.equal(o, want)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("nq", [1, 5, 150])
def test_a_captured_step(dtype, nq):
    """Rotate, append, attend, add up the weights, evict and read back in one graph,
    over inputs that change between replays: as the eager calls, bit by bit."""
    B, hq, hkv, dim, bs, room, keep = 3, 8, 2, 64, 16, 640, 200
    r = kvq.Rope.make(dim)

    def state(seed):
        c, _ = filled(seed, [room] * B, hkv, dim, bs)
        into, _ = filled(seed + 1, [keep] * B, hkv, dim, bs)
        x = rand(seed + 2, B * nq, hq + 2 * hkv, dim, dtype=dtype)
        lens = ints([seed % 300 + nq, 7 + nq, 450])
        return [c.k_codes, c.k_scales, c.v_codes, c.v_scales, c.block_table, into.k_codes,
                into.k_scales, into.v_codes, into.v_scales, into.block_table, x, lens]

    def step(s):
        c, into = kvq.B8Cache.wrap(*s[:5]), kvq.B8Cache.wrap(*s[5:10])
        x, lens = s[10:]
        cu = torch.arange(0, B * nq + 1, nq, dtype=torch.int32, device="cuda")
        start = lens - nq
        pos = (start[:, None] + torch.arange(nq, dtype=torch.int32, device="cuda")).contiguous()
        kw = dict(cu_q=cu, max_q=nq) if nq > 1 else {}
        q, _ = kvq.rope(x[:, :hq], None, pos.view(-1), r)
        kv = x.view(B, nq, hq + 2 * hkv, dim)
        kvq.b8_append(c, kv[:, :, hq:hq + hkv], kv[:, :, hq + hkv:], start, rope=r)
        out, lse = kvq.b8_attn(c, q, lens, room, 0.125, return_lse=True, **kw)
        m = torch.zeros((B, hkv, room), device="cuda")
        kvq.b8_attn_mass(c, q, lse, lens, room, 0.125, m, **kw)
        ev = kvq.b8_evict(c, into, m, lens, room, keep, recent=20, sinks=2)
        return (out, lse, m, *ev, *kvq.b8_gather(into, torch.zeros_like(lens), ev[0], keep, dtype))

    seeds = (201, 305, 411)
    want = [[t.clone() for t in step(state(s))] for s in seeds]
    held = state(seeds[0])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step(held)
        st.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=st):
            got = step(held)
        for seed, w in zip(seeds, want):
            for t, new in zip(held, state(seed)):
                t.copy_(new)
            gr.replay()
            gr.replay()  # the same tokens again, over their own codes
            st.synchronize()
            for i, (a, b) in enumerate(zip(got, w)):
                assert torch.equal(a, b), i


def test_refusals_on_the_device():
    c, _ = filled(141, [64], 1, 64, 16)
    q = rand(142, 1, 2, 64)
    with pytest.raises(ValueError):
        kvq.b8_attn(c, q, ints([64]).cpu(), 64, 0.1)
    with pytest.raises(ValueError):
        kvq.b8_attn(c, q, ints([64]), 64, 0.1, out=torch.empty_like(q).half())
    with pytest.raises(TypeError):
        kvq.b8_attn(c, q.half(), ints([64]), 64, 0.1)
    with pytest.raises(kvq.KVQError) as e:
        kvq.b8_attn(c, q, ints([64]), 64, float("nan"))
    assert e.value.status == kvq.KVQ_ERR_INVALID_ARG
    with pytest.raises(kvq.KVQError):
        kvq.b8_evict(c, c, torch.zeros((1, 1, 64), device="cuda"), ints([64]), 64, 65)
    e = kvq.b8_attn(c, q[:0], ints([]), 64, 0.1)
    assert e.shape == (0, 2, 64)
