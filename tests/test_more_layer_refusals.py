"""Rotary positions, the rotating append, the 4-bit cache and the norms around
a block without a GPU: what they refuse, by the C ABI (each call below is
refused, or has no rows) and by the binding, and pins of their oracle."""

import math

import numpy as np
import pytest
import torch

import oracle.layer as OL
import tenant_linear_layers_amd as T

A, B, C, D, E, F, G, H = (0x1000000 * i for i in range(1, 9))   # never dereferenced


# ------------------------------------------------------------------ C ABI
def test_rotary_argument_errors():
    f = T.lib().bitdelta_rotary

    def call(x=A, st=(1024, 128), pos=B, table=C, length=100, rot=128, tokens=3, heads=8, dim=128,
             out=D, ost=(1024, 128)):
        return f(x, *st, pos, table, length, rot, 0, tokens, heads, dim, out, *ost, None)

    assert call(tokens=0) == 0 and call(tokens=0, x=None, out=None) == 0
    for bad in (dict(tokens=-1), dict(heads=0), dict(heads=65537), dict(dim=65538, rot=2),
                dict(dim=1, rot=2), dict(rot=0), dict(rot=-2), dict(rot=3), dict(rot=130),
                dict(length=0), dict(length=1 << 31), dict(length=1 << 30, rot=1024, dim=1024),
                dict(st=(-1, 128)), dict(st=(1024, -128)), dict(ost=(-1, 128)),
                dict(ost=(1024, 1 << 40))):
        assert call(**bad) == 2, bad
    # rows of out that lie over one another
    for ost in ((0, 128), (1024, 0), (1024, 64), (1023, 128), (128, 383), (64, 1024)):
        assert call(ost=ost) == 2, ost
    for bad in (dict(x=None), dict(pos=None), dict(table=None), dict(out=None)):
        assert call(**bad) == 1, bad
    for bad in (dict(x=A + 1), dict(out=D + 1), dict(pos=B + 2), dict(table=C + 2)):
        assert call(**bad) == 3, bad
    for bad in (dict(out=A, ost=(2048, 128)), dict(out=A + 256), dict(out=B), dict(out=C + 64),
                dict(out=A, ost=(128, 384))):
        assert call(**bad) == 9, bad


def test_rotary_table_argument_errors():
    f = T.lib().bitdelta_rotary_table

    def call(freq=A, pairs=64, first=0, length=10, table=B):
        return f(freq, pairs, first, length, 1.0, table, None)

    assert call(length=0) == 0 and call(length=0, freq=None) == 0
    for bad in (dict(pairs=0), dict(pairs=32769), dict(first=-1), dict(first=1 << 31),
                dict(length=-1), dict(length=1 << 31), dict(length=1 << 30, pairs=32768)):
        assert call(**bad) == 2, bad
    assert call(freq=None) == 1 and call(table=None) == 1
    assert call(freq=A + 4) == 3 and call(table=B + 4) == 3
    assert call(table=A) == 9 and call(table=A + 504) == 9


def test_kv_append_argument_errors():
    f = T.lib().bitdelta_kv_append

    def call(q=A, qs=(2048, 128), k=A + 1024, ks=(2048, 128), v=A + 1536, vs=(2048, 128), pos=B,
             table=B + 65536, length=50, rot=64, slots=B + 4096, tokens=3, heads=4, kv_heads=2,
             dim=128, pages=2, page=16, bits=16, kc=C, vc=D, ksc=None, vsc=None, out=E):
        return f(q, *qs, k, *ks, v, *vs, pos, table, length, rot, 0, slots, tokens, heads,
                 kv_heads, dim, pages, page, bits, kc, vc, ksc, vsc, out, None)

    assert call(tokens=0) == 0 and call(tokens=0, q=None, k=None, out=None) == 0
    for bad in (dict(tokens=-1), dict(heads=0), dict(heads=1025), dict(kv_heads=0), dict(dim=96),
                dict(page=20), dict(pages=0), dict(bits=5), dict(bits=0), dict(bits=2),
                dict(rot=0), dict(rot=130), dict(rot=63), dict(length=0), dict(qs=(-1, 128)),
                dict(ks=(2048, -1)), dict(vs=(1 << 41, 128))):
        assert call(**bad) == 2, bad
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(pos=None), dict(table=None),
                dict(slots=None), dict(kc=None), dict(vc=None), dict(out=None), dict(bits=8),
                dict(bits=4), dict(bits=4, ksc=F), dict(ksc=F, vsc=G), dict(bits=8, vsc=F)):
        assert call(**bad) == 1, bad
    for bad in (dict(q=A + 1), dict(pos=B + 2), dict(table=B + 65538), dict(slots=B + 4097),
                dict(kc=C + 8), dict(out=E + 1), dict(bits=4, ksc=F + 8, vsc=G)):
        assert call(**bad) == 3, bad
    for bad in (dict(out=A), dict(out=A + 1500), dict(out=B), dict(out=B + 65540),
                dict(out=B + 4100), dict(out=C), dict(out=D + 64), dict(kc=D), dict(kc=A),
                dict(kc=B), dict(kc=B + 65536), dict(vc=B + 65536 - 4096),
                dict(bits=4, ksc=F, vsc=F + 64), dict(bits=4, ksc=F, vsc=E),
                dict(bits=8, ksc=F, vsc=C + 16)):
        assert call(**bad) == 9, bad


def test_kv_4bit_argument_errors():
    w, r = T.lib().bitdelta_kv_write_4bit, T.lib().bitdelta_kv_read_4bit

    def wr(k=A, v=A + 1024, st=(2048, 128, 2048, 128), slots=B, tokens=3, heads=4, dim=128,
           pages=2, page=16, kc=C, vc=D, ks=G, vs=H):
        return w(k, v, *st, slots, tokens, heads, dim, pages, page, kc, vc, ks, vs, None)

    def rd(slots=B, tokens=3, heads=4, dim=128, pages=2, page=16, kc=C, vc=D, ks=G, vs=H, k=E,
           v=F):
        return r(slots, tokens, heads, dim, pages, page, kc, vc, ks, vs, k, v, None)

    for f in (wr, rd):
        assert f(tokens=0) == 0 and f(tokens=0, slots=None) == 0
        assert f(tokens=-1) == 2 and f(dim=96) == 2 and f(page=8) == 2 and f(pages=0) == 2
        assert f(heads=0) == 2 and f(heads=1025) == 2
        assert f(slots=None) == 1 and f(kc=None) == 1 and f(ks=None) == 1 and f(vs=None) == 1
        assert f(kc=C + 8) == 3 and f(slots=B + 2) == 3 and f(ks=G + 4) == 3 and f(vs=H + 8) == 3
    # a row of 128 dims: 64 bytes and 4 of scales
    assert wr(vc=C + 2 * 4 * 16 * 64 - 16) == 9 and wr(vs=G + 2 * 4 * 16 * 4 - 16) == 9
    assert wr(kc=A) == 9 and wr(ks=C + 16) == 9 and wr(st=(-1, 128, 2048, 128)) == 2
    assert rd(k=C) == 9 and rd(v=E + 256) == 9 and rd(k=G + 496) == 9 and rd(k=E + 8) == 3


def test_paged_attention_4bit_argument_errors():
    f = T.lib().bitdelta_paged_attention_4bit

    def call(q=A, st=(1024, 128), kc=B, vc=C, ks=G, vs=H, table=D, cu=D + 4096, kv=D + 8192,
             tokens=5, seqs=2, max_q=4, heads=8, kv_heads=2, dim=128, pages=4, page=16, width=3,
             scale=1.0, window=0, out=E, ws=F, wn=1 << 40):
        return f(q, *st, kc, vc, ks, vs, table, cu, kv, tokens, seqs, max_q, heads, kv_heads,
                 dim, pages, page, width, scale, window, out, ws, wn, None)

    assert call(tokens=0) == 0 and call(seqs=0) == 0 and call(max_q=0, q=None) == 0
    for bad in (dict(tokens=-1), dict(heads=9), dict(heads=130, kv_heads=2), dict(dim=80),
                dict(page=20), dict(pages=0), dict(width=-1), dict(window=-1), dict(scale=0.0),
                dict(scale=math.nan), dict(tokens=1 << 29), dict(st=(-8, 128))):
        assert call(**bad) == 2, bad
    for bad in (dict(q=None), dict(kc=None), dict(table=None), dict(out=None), dict(ks=None),
                dict(vs=None), dict(ks=None, vs=None)):
        assert call(**bad) == 1, bad
    for bad in (dict(q=A + 1), dict(kc=B + 8), dict(ks=G + 4), dict(vs=H + 2), dict(out=E + 8),
                dict(ws=F + 4)):
        assert call(**bad) == 3, bad
    for bad in (dict(out=A), dict(out=B), dict(out=C + 64), dict(out=D), dict(out=G),
                dict(out=H + 4 * 2 * 16 * 4 - 16)):
        assert call(**bad) == 9, bad


def test_rms_norm_block_argument_errors():
    f = T.lib().bitdelta_rms_norm_block

    def call(x=A, xs=64, post=B, gate=C, gs=64, alpha=1.0, r=D, rs=64, w=E, rows=4, cols=64, h=F,
             y=G):
        return f(x, xs, post, gate, gs, alpha, r, rs, w, 1e-5, rows, cols, h, y, None)

    assert call(rows=0) == 0 and call(rows=0, x=None, y=None) == 0
    for bad in (dict(rows=-1), dict(cols=0), dict(rows=1 << 31), dict(cols=(1 << 30) + 1),
                dict(rows=1 << 20, cols=1 << 21), dict(xs=-1), dict(rs=-64), dict(gs=-1),
                dict(alpha=math.inf), dict(alpha=math.nan)):
        assert call(**bad) == 2, bad
    for bad in (dict(x=None), dict(r=None), dict(w=None), dict(h=None), dict(y=None)):
        assert call(**bad) == 1, bad
    for bad in (dict(x=A + 1), dict(post=B + 1), dict(gate=C + 1), dict(r=D + 1), dict(w=E + 1),
                dict(h=F + 1), dict(y=G + 1)):
        assert call(**bad) == 3, bad
    for bad in (dict(y=A), dict(y=B), dict(y=C + 2), dict(y=D), dict(y=E), dict(y=F + 8),
                dict(h=A), dict(h=D), dict(y=C + 126, gs=0)):
        assert call(**bad) == 9, bad


# ------------------------------------------------------------------ binding
def test_binding_refuses_host_tensors_and_non_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.ones(64, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    k, table = x.view(4, 1, 64), torch.zeros(8, 32, 2)
    c = torch.zeros(2, 1, 16, 32, dtype=torch.uint8).view(torch.float4_e2m1fn_x2)
    s = torch.zeros(2, 1, 16, 2, dtype=torch.uint8).view(torch.float8_e8m0fnu)
    for call in (lambda: T.rms_norm_block(x, x, w, w, 1e-5), lambda: T.rotary(k, i, table),
                 lambda: T.kv_append(k, k, k, i, table, i, c, c, s, s),
                 lambda: T.kv_write(k, k, i, c, c, s, s), lambda: T.kv_read(i, c, c, s, s),
                 lambda: T.paged_attention(k, c, c, i.view(4, 1), torch.zeros(5), i, 1, s, s)):
        with pytest.raises(ValueError, match="device"):
            call()
    with pytest.raises(TypeError):
        T.rotary([1.0], i, table)
    with pytest.raises(TypeError):
        T.rotary_table(torch.zeros(4), 8)


def test_rotary_frequencies():
    """The plain ones, and each way of stretching them against its definition."""
    f, m = T.rotary_frequencies(8)
    assert m == 1.0 and f.dtype == torch.float64
    assert np.allclose(f, [1.0, 10.0 ** -1, 10.0 ** -2, 10.0 ** -3], rtol=1e-14)
    assert np.allclose(T.rotary_frequencies(8, factor=4.0)[0], f.numpy() / 4, rtol=1e-14)
    g, m = T.rotary_frequencies(128, 500000.0, 8.0, "base")
    p, _ = T.rotary_frequencies(128, 500000.0)
    assert m == 1.0 and g[0] == 1.0 and abs(g[-1] * 8 / p[-1] - 1) < 1e-12
    for method in ("ramp", "smooth"):
        g, m = T.rotary_frequencies(128, 10000.0, 16.0, method, original_length=4096)
        p, _ = T.rotary_frequencies(128)
        turns = 4096 * p / (2 * math.pi)
        stretched = p / g
        assert bool((stretched[turns > 40] == 1).all())
        assert np.allclose(stretched[turns < 0.8], 16.0, rtol=1e-12)
        assert bool((stretched[1:] >= stretched[:-1] - 1e-12).all())   # and rising between
        assert abs(m - (0.1 * math.log(16) + 1 if method == "ramp" else 1.0)) < 1e-15
    assert np.array_equal(T.rotary_frequencies(64, factor=1.0, method="smooth",
                                               original_length=4096)[0],
                          T.rotary_frequencies(64)[0])
    for bad in (dict(rot=7), dict(rot=0), dict(rot=8, base=0.0), dict(rot=8, factor=-1.0),
                dict(rot=8, method="other"), dict(rot=8, factor=2.0, method="ramp"),
                dict(rot=8, method="smooth", original_length=64, fast=1.0, slow=1.0),
                dict(rot=2, factor=2.0, method="base")):
        with pytest.raises(ValueError):
            T.rotary_frequencies(**bad)


# ------------------------------------------------------------------ oracle
def test_oracle_e2m1_codes_and_borders():
    for c in range(16):
        v = (-1.0 if c & 8 else 1.0) * OL.E2M1[c & 7]
        assert OL.e2m1_codes(np.array([v]))[0] == c or (c == 8 and v == 0)
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    assert list(OL.e2m1_codes(ties)) == [0, 2, 2, 4, 4, 6, 6]
    assert list(OL.e2m1_codes(np.nextafter(ties, 9))) == [1, 2, 3, 4, 5, 6, 7]
    assert list(OL.e2m1_codes(np.nextafter(ties, 0))) == [0, 1, 2, 3, 4, 5, 6]


def test_oracle_4bit_groups():
    x = np.zeros((1, 96))
    x[0, 0] = 6.0 * 2.0 ** 5
    x[0, 33] = np.nextafter(6.0 * 2.0 ** 5, np.inf)
    x[0, 70] = np.nan
    q, s = OL.quantise4(x)
    assert q.shape == (1, 48) and list(s[0]) == [132, 133, 255]
    back = OL.dequantise4(q, s)
    assert back[0, 0] == 192.0 and back[0, 33] == 192.0 and np.isnan(back[0, 64:]).all()
    assert np.all(back[0, 1:32] == 0)
    # within the grid a value is at most half a step off: 2^-2 of it, a quarter of the scale
    g = np.random.default_rng(3).normal(size=(50, 64)) * np.exp2(np.arange(50) - 25.0)[:, None]
    q, s = OL.quantise4(g)
    step = np.repeat(np.exp2(s.astype(float) - 127), 32, axis=1)
    assert np.all(np.abs(OL.dequantise4(q, s) - g) <= np.maximum(np.abs(g) / 4, step / 4))


def test_oracle_rotary():
    g = np.random.default_rng(4)
    x, a = g.normal(size=(5, 2, 12)), g.uniform(-9, 9, size=(5, 4))
    out = OL.rotary(x, a)
    assert np.array_equal(out[..., 8:], x[..., 8:])
    assert np.allclose(out[:, :, 1], x[:, :, 1] * np.cos(a[:, None, 1]) -
                       x[:, :, 5] * np.sin(a[:, None, 1]))
    assert np.allclose(out[:, :, 5], x[:, :, 5] * np.cos(a[:, None, 1]) +
                       x[:, :, 1] * np.sin(a[:, None, 1]))
    order = [0, 4, 1, 5, 2, 6, 3, 7, 8, 9, 10, 11]
    assert np.allclose(OL.rotary(x[..., order], a, True), out[..., order])
