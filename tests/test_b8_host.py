"""Host-side checks of the rotary positions and of the block-scaled 8-bit cache
(no GPU): frequencies, argument validation of every call before any launch."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

from hadamard_rotated_bit_fwht_b200 import build, kvq

INVALID, UNSUPPORTED, WORKSPACE = (kvq.KVQ_ERR_INVALID_ARG, kvq.KVQ_ERR_UNSUPPORTED,
                                   kvq.KVQ_ERR_WORKSPACE)


@pytest.fixture(scope="module")
def L():
    build.build()
    return kvq.lib()


@pytest.fixture(scope="module")
def p16():
    buf = (C.c_uint8 * 8192)()
    p16.keep = buf
    return (C.addressof(buf) + 15) // 16 * 16


def cache_desc(p, **kw):
    d = dict(hkv=2, dim=128, bs=16, nb=8, seqs=2, cols=4)
    d.update(kw)
    return kvq.B8CacheDesc(p, p, p, p, d["hkv"], d["dim"], d["bs"], d["nb"], p, d["seqs"],
                           d["cols"])


def heads(p, n=2, token=256, head=128):
    return kvq.HeadsDesc(p, token, head, n)


@pytest.mark.parametrize("rot", [2, 16, 64, 128])
def test_frequencies(L, rot):
    base, s, trained = 10000.0, 8.0, 4096.0
    i = np.arange(rot // 2)
    plain = base ** (-2.0 * i / rot)

    def got(**kw):
        r = kvq.Rope.make(rot, base, device="cpu", **kw)
        return r.inv_freq.numpy(), r.factor

    f, m = got()
    np.testing.assert_allclose(f, plain, rtol=1e-14)
    assert m == 1.0
    f, m = got(scaling="linear", scale=s)
    np.testing.assert_allclose(f, plain / s, rtol=1e-14)
    f, m = got(scaling="ntk", scale=s)
    b2 = base * s ** (rot / (rot - 2)) if rot > 2 else base
    np.testing.assert_allclose(f, b2 ** (-2.0 * i / rot), rtol=1e-13)
    if rot > 2:  # the lowest frequency is the linear one's
        np.testing.assert_allclose(f[-1], plain[-1] / s, rtol=1e-13)
    f, m = got(scaling="yarn", scale=s, trained_len=trained)
    for x, y in zip(f, plain):
        turns = trained * y / (2 * math.pi)
        keep = min(max((turns - 1) / 31, 0), 1)
        assert math.isclose(x, y / s * (1 - keep) + y * keep, rel_tol=1e-13)
    assert math.isclose(m, 0.1 * math.log(s) + 1, rel_tol=1e-6)


def test_yarn_ramps_differ_between_their_ends_only():
    """The ramp in turns, which is offered, and the one in the pair's index: equal
    outside, different inside, as the header says."""
    rot, base, s, trained = 128, 10000.0, 8.0, 4096.0
    got = kvq.Rope.make(rot, base, scaling="yarn", scale=s, trained_len=trained, device="cpu")
    i = np.arange(rot // 2)
    plain = base ** (-2.0 * i / rot)
    index = lambda turns: rot * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))
    low, high = math.floor(index(32.0)), math.ceil(index(1.0))
    ramp = np.clip((i - low) / (high - low), 0, 1)
    by_index = plain * (1 - ramp) + plain / s * ramp
    f = got.inv_freq.numpy()
    out = (i <= low) | (i >= high)
    np.testing.assert_allclose(f[out], by_index[out], rtol=1e-13)
    assert (np.abs(f / by_index - 1)[low + 2:high - 1] > 1e-2).all()
    # such a model's own table
    own = kvq.Rope(torch.from_numpy(by_index), False, got.factor)
    assert own.inv_freq.dtype == torch.float64 and own.inv_freq.numel() == rot // 2


def test_frequency_refusals():
    for kw in (dict(rot_dim=7), dict(rot_dim=0), dict(rot_dim=16, base=-1.0),
               dict(rot_dim=16, scaling="linear", scale=0.5),
               dict(rot_dim=16, scaling="yarn", scale=2.0),
               dict(rot_dim=16, scaling="yarn", scale=2.0, trained_len=10, beta_fast=1.0),
               dict(rot_dim=16, base=float("nan"))):
        with pytest.raises(kvq.KVQError) as e:
            kvq.Rope.make(device="cpu", **kw)
        assert e.value.status == INVALID
    with pytest.raises(ValueError):
        kvq.Rope.make(16, scaling="cubic", device="cpu")


def test_rope_refusals(L, p16):
    spec = lambda rot=128, factor=1.0, p=p16: kvq.RopeDesc(p, rot, 0, factor)
    x = heads(p16)

    def call(s=None, dtype=1, dim=128, n=1, pos=p16, q=x, qo=x, k=x, ko=x):
        ref = lambda h: None if h is None else C.byref(h)
        return L.kvq_rope(C.byref(s or spec()), dtype, dim, n, pos, 0, ref(q), ref(qo), ref(k),
                          ref(ko), None)

    assert call(n=0) == kvq.KVQ_OK
    assert call(n=-1) == INVALID
    assert call(dtype=5) == INVALID
    assert call(pos=None) == INVALID
    assert call(q=None) == INVALID
    assert call(ko=None) == INVALID
    assert call(s=spec(p=None)) == INVALID
    assert call(s=spec(rot=144)) == INVALID
    assert call(s=spec(rot=24)) == UNSUPPORTED
    assert call(s=spec(factor=float("inf"))) == INVALID
    assert call(dim=520, s=spec()) == UNSUPPORTED
    assert call(q=heads(p16 + 2)) == INVALID
    assert call(q=heads(p16, token=250)) == INVALID
    assert call(qo=heads(p16, n=3)) == INVALID
    assert call(qo=heads(p16, token=512)) == INVALID  # in place with other strides


def test_rope_refuses_outputs_that_share_elements(L, p16):
    spec = kvq.RopeDesc(p16, 64, 0, 1.0)
    x = heads(p16 + 4096)

    def call(out, n=4, src=x):
        return L.kvq_rope(C.byref(spec), 1, 128, n, p16, 0, C.byref(src), C.byref(out), None, None,
                          None)

    for token, head in ((0, 128), (256, 0), (256, 64), (120, 512), (256, 256), (-64, 512), (512, -64)):
        o = heads(p16, token=token, head=head)
        assert call(o) == INVALID, (token, head)
        assert call(o, src=o) == INVALID, (token, head)  # in place
    if not torch.cuda.is_available():  # fine, as far as the launch
        for o in (heads(p16, token=256, head=128), heads(p16, token=128, head=512),
                  heads(p16, token=-256, head=128)):
            assert call(o) == kvq.KVQ_ERR_CUDA
        # one token, one head: their strides mean nothing
        assert call(heads(p16, token=0, head=128), n=1) == kvq.KVQ_ERR_CUDA
        one = heads(p16 + 4096, n=1)
        assert call(heads(p16, n=1, token=256, head=0), src=one) == kvq.KVQ_ERR_CUDA
        # inputs may be broadcast
        assert call(heads(p16), src=heads(p16 + 4096, token=0, head=0)) == kvq.KVQ_ERR_CUDA


def test_cache_refusals(L, p16):
    x = heads(p16)

    def call(d, k=x, v=x, dtype=1, batch=1, t=1, start=p16, rope=None):
        return L.kvq_b8_append(C.byref(d), C.byref(k), C.byref(v), dtype, batch, t, start, None,
                               None if rope is None else C.byref(rope), None, None)

    d = cache_desc(p16)
    assert call(d, batch=0) == kvq.KVQ_OK
    assert call(d, t=0) == kvq.KVQ_OK
    assert call(d, batch=3) == INVALID
    assert call(d, dtype=2) == INVALID
    assert call(d, start=None) == INVALID
    assert call(d, k=heads(p16, n=3)) == INVALID
    assert call(d, rope=kvq.RopeDesc(p16, 8, 0, 1.0)) == UNSUPPORTED
    assert call(d, rope=kvq.RopeDesc(p16, 256, 0, 1.0)) == INVALID
    for kw, st in ((dict(dim=96), UNSUPPORTED), (dict(bs=24), UNSUPPORTED), (dict(nb=0), INVALID),
                   (dict(cols=0), INVALID), (dict(seqs=0), INVALID), (dict(hkv=0), INVALID),
                   (dict(nb=1 << 26), UNSUPPORTED), (dict(cols=1 << 28), UNSUPPORTED)):
        assert call(cache_desc(p16, **kw)) == st, kw
    bad = cache_desc(p16)
    bad.k_scales = None
    assert call(bad) == INVALID
    bad = cache_desc(p16 + 8)
    assert call(bad) == INVALID

    def gather(d, batch=1, count=1, out=p16, dtype=1):
        return L.kvq_b8_gather(C.byref(d), batch, p16, p16, count, dtype, out, p16, None)

    assert gather(d, count=0) == kvq.KVQ_OK
    assert gather(d, count=-1) == INVALID
    assert gather(d, batch=3) == INVALID
    assert gather(d, out=p16 + 4) == INVALID
    assert gather(d, dtype=9) == INVALID


def queries(p, hq=4, dtype=1, batch=2, total=2, max_q=1, cu=None, lens=0, max_len=64, scale=0.1):
    return kvq.B8QueriesDesc(heads(p, n=hq), dtype, batch, total, max_q, cu,
                             p if lens == 0 else lens, max_len, scale)


def test_attention_refusals(L, p16):
    d = cache_desc(p16)

    def call(q, d=d, out=p16, ws=None, n=0):
        return L.kvq_b8_attn(C.byref(d), C.byref(q), out, None, ws, n, None)

    assert call(queries(p16, batch=0, total=0)) == kvq.KVQ_OK
    assert call(queries(p16, total=0, cu=p16)) == kvq.KVQ_OK
    for kw in (dict(hq=3), dict(dtype=7), dict(batch=3, total=3), dict(total=3),
               dict(max_len=-1), dict(scale=float("nan")), dict(lens=None), dict(max_q=-1, cu=p16)):
        assert call(queries(p16, **kw)) == INVALID, kw
    assert call(queries(p16), out=None) == INVALID
    assert call(queries(p16), out=p16 + 8) == INVALID
    big = cache_desc(p16, cols=2048)
    q = queries(p16, max_len=32768)
    need = L.kvq_b8_attn_workspace(C.byref(big), 1, 4, 2, 1, 32768)
    assert need > 0
    assert call(q, d=big) == WORKSPACE
    assert call(q, d=big, ws=p16, n=need - 1) == WORKSPACE
    assert call(q, d=big, ws=p16 + 4, n=need) == WORKSPACE
    assert L.kvq_b8_attn_workspace(C.byref(big), 1, 3, 2, 1, 32768) == 0
    assert L.kvq_b8_attn_workspace(C.byref(cache_desc(p16, dim=80)), 1, 4, 2, 1, 32768) == 0
    wide = queries(p16, batch=2, total=1 << 30, max_q=(1 << 31) - 1, cu=p16)
    assert call(wide) == UNSUPPORTED


def test_attention_refuses_to_write_over_its_queries(L, p16):
    d, q = cache_desc(p16), queries(p16 + 4096)

    def call(out):
        return L.kvq_b8_attn(C.byref(d), C.byref(q), out, None, None, 0, None)

    assert call(p16 + 4096) == INVALID
    if not torch.cuda.is_available():  # elsewhere: as far as the launch
        assert call(p16) == kvq.KVQ_ERR_CUDA


def test_mass_and_evict_refusals(L, p16):
    d = cache_desc(p16)

    def mass(q, lse=p16, m=p16, stride=64):
        return L.kvq_b8_attn_mass(C.byref(d), C.byref(q), lse, m, stride, None)

    assert mass(queries(p16, batch=0, total=0)) == kvq.KVQ_OK
    assert mass(queries(p16, max_len=0)) == kvq.KVQ_OK
    assert mass(queries(p16), lse=None) == INVALID
    assert mass(queries(p16), m=None) == INVALID
    assert mass(queries(p16), stride=63) == INVALID
    assert mass(queries(p16, hq=5)) == INVALID

    def evict(dst=d, batch=1, max_len=64, keep=8, recent=2, sinks=2, ms=64, mo=8, m=p16):
        return L.kvq_b8_evict(C.byref(d), C.byref(dst), batch, p16, max_len, m, ms, keep, recent,
                              sinks, p16, p16, p16, mo, None)

    assert evict(batch=0) == kvq.KVQ_OK
    for kw in (dict(keep=0), dict(recent=7), dict(sinks=-1), dict(recent=-1), dict(ms=63),
               dict(mo=7), dict(keep=65, mo=65), dict(batch=3), dict(m=None),
               dict(dst=cache_desc(p16, hkv=1)), dict(dst=cache_desc(p16, dim=64))):
        assert evict(**kw) == INVALID, kw


def test_evict_outputs_are_no_inputs(L, p16):
    """Each refusal alone: pointers that differ, then one shared."""
    d = cache_desc(p16)
    at = {n: C.c_void_p((i + 2) * 4096) for i, n in enumerate(("lens", "mass", "new", "kept", "out"))}

    def evict(ms=64, mo=8, **kw):
        p = {**at, **kw}
        return L.kvq_b8_evict(C.byref(d), C.byref(d), 1, p["lens"], 64, p["mass"], ms, 8, 2, 2,
                              p["new"], p["kept"], p["out"], mo, None)

    for kw in (dict(new=at["lens"]), dict(out=at["mass"]), dict(mass=None), dict(lens=None),
               dict(new=None), dict(kept=None), dict(out=None), dict(ms=63), dict(mo=7)):
        assert evict(**kw) == INVALID, kw


def test_each_refusal_of_evict_alone(L):
    """Pointers and caches that are all fine, then one argument that is not."""
    P = lambda i: (i + 1) << 20

    def cache(at, **kw):
        d = cache_desc(P(0), **kw)
        d.k_codes, d.k_scales, d.v_codes, d.v_scales, d.block_table = (P(at + i) for i in range(5))
        return d

    base = dict(src=cache(0), dst=cache(5), batch=2, lens=P(10), max_len=64, mass=P(11), ms=64,
                keep=8, recent=2, sinks=2, new=P(12), kept=P(13), out=P(14), mo=8)

    def evict(**kw):
        a = {**base, **kw}
        return L.kvq_b8_evict(C.byref(a["src"]), C.byref(a["dst"]), a["batch"], a["lens"], a["max_len"],
                              a["mass"], a["ms"], a["keep"], a["recent"], a["sinks"], a["new"],
                              a["kept"], a["out"], a["mo"], None)

    if not torch.cuda.is_available():  # all fine: as far as the launch
        assert evict() == kvq.KVQ_ERR_CUDA
        # side by side is fine: 2 sequences, 2 heads
        assert evict(new=P(10) + 8, kept=P(11) + 4 * (3 * 64 + 64),
                     out=P(13) + 4 * 4 * 8) == kvq.KVQ_ERR_CUDA
    assert evict(batch=0) == kvq.KVQ_OK
    for kw in (dict(batch=-1), dict(batch=3), dict(src=cache(0, seqs=1)), dict(dst=cache(5, seqs=1)),
               dict(max_len=-1), dict(keep=0), dict(recent=-1), dict(sinks=-1),
               dict(recent=7), dict(sinks=7), dict(recent=(1 << 31) - 1, sinks=(1 << 31) - 1),
               dict(keep=65, mo=65), dict(dst=cache(5, hkv=1)), dict(dst=cache(5, dim=64)),
               dict(lens=None), dict(mass=None), dict(new=None), dict(kept=None), dict(out=None),
               dict(ms=63), dict(mo=7),
               # outputs that are inputs or one another, whole or in part
               dict(new=P(10)), dict(kept=P(10)), dict(out=P(10)), dict(new=P(10) + 4),
               dict(kept=P(10) - 4 * (4 * 8 - 1)), dict(new=P(11)), dict(kept=P(11)),
               dict(out=P(11)), dict(out=P(11) + 4 * 255), dict(out=P(11) - 4 * 31),
               dict(new=P(13) + 4 * 31), dict(kept=P(14)), dict(out=P(12) + 4)):
        assert evict(**kw) == INVALID, kw
    for kw in (dict(src=cache(0, dim=96), dst=cache(5, dim=96)), dict(dst=cache(5, bs=24))):
        assert evict(**kw) == UNSUPPORTED, kw


def test_evict_onto_its_own_blocks(L):
    P = lambda i: (i + 1) << 20

    def cache(*at):
        d = cache_desc(P(0))
        d.k_codes, d.k_scales, d.v_codes, d.v_scales, d.block_table = (P(i) for i in at)
        return d

    def evict(src, dst, batch=1):
        return L.kvq_b8_evict(C.byref(src), C.byref(dst), batch, P(20), 64, P(21), 64, 8, 2, 2, P(22),
                              P(23), P(24), 8, None)

    src = cache(0, 1, 2, 3, 4)
    assert evict(src, src, batch=0) == kvq.KVQ_OK
    assert evict(src, src) == INVALID
    for shared in range(4):  # any plane in common
        at = [0 + i if i == shared else 10 + i for i in range(4)] + [4]
        assert evict(src, cache(*at)) == INVALID, shared
    if not torch.cuda.is_available():  # another table, or other planes: as far as the launch
        assert evict(src, cache(0, 1, 2, 3, 9)) == kvq.KVQ_ERR_CUDA
        assert evict(src, cache(10, 11, 12, 13, 4)) == kvq.KVQ_ERR_CUDA


def test_bindings_check_shapes_first():
    z = lambda *s, t=torch.float32: torch.zeros(s, dtype=t)
    with pytest.raises(ValueError, match="codes"):
        kvq.B8Cache.wrap(z(4, 2, 16, t=torch.int8), z(4, 2), z(4, 2, 16, t=torch.int8), z(4, 2),
                         z(1, 4, t=torch.int32))
    with pytest.raises(ValueError, match="k_codes"):
        kvq.B8Cache.wrap(z(4, 2, 16, 64), z(4, 2), z(4, 2, 16, 64), z(4, 2),
                         z(1, 4, t=torch.int32))
    c = kvq.B8Cache(4, 2, 16, 64, z(1, 4, t=torch.int32), device="cpu")
    assert c.capacity == 64
    i = z(1, t=torch.int32)
    with pytest.raises(ValueError, match="q must be"):
        kvq.b8_attn(c, z(1, 3, 64), i, 16, 0.1)
    with pytest.raises(ValueError, match="one query"):
        kvq.b8_attn(c, z(2, 4, 64), i, 16, 0.1)
    with pytest.raises(ValueError, match="max_q"):
        kvq.b8_attn(c, z(2, 4, 64), i, 16, 0.1, cu_q=z(2, t=torch.int32))
    with pytest.raises(ValueError, match="seq_lens"):
        kvq.b8_attn(c, z(1, 4, 64), i.long(), 16, 0.1)
    with pytest.raises(ValueError, match="mass"):
        kvq.b8_attn_mass(c, z(1, 4, 64), z(1, 4), i, 16, 0.1, z(1, 2, 15))
    with pytest.raises(ValueError, match="mass"):
        kvq.b8_evict(c, c, z(1, 2, 15), i, 16, 4)
    with pytest.raises(ValueError, match="same"):
        kvq.b8_append(c, z(1, 1, 2, 64), z(1, 2, 2, 64), i)
    with pytest.raises(ValueError, match="stride"):  # tokens at two strides
        kvq.rope(z(3, 4, 2, 64)[:, :3], None, z(9, t=torch.int32), kvq.Rope(
            z(16, t=torch.float64)))
    with pytest.raises(ValueError, match="inv_freq"):
        kvq.rope(z(3, 2, 64), None, z(3, t=torch.int32), kvq.Rope(z(16)))
    with pytest.raises(TypeError):
        kvq.b8_gather(c, i, i, 4, torch.float16)
    with pytest.raises(TypeError):
        kvq.b8_attn(c, z(1, 4, 64, t=torch.float16), i, 16, 0.1)
    with pytest.raises(TypeError):
        kvq.b8_attn(c, None, i, 16, 0.1)
    with pytest.raises(TypeError):
        kvq.b8_attn(c, z(1, 4, 64), i, 16.5, 0.1)
    with pytest.raises(ValueError, match="32 bits"):
        kvq.b8_attn(c, z(1, 4, 64), i, 1 << 31, 0.1)
