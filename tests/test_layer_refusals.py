"""The decoder-layer operators without a GPU: what they refuse, by the C ABI
(no call below reaches the runtime: each is refused, or has no rows) and by the
binding, and pins of their float64 oracle."""

import math

import numpy as np
import pytest
import torch

import oracle.layer as OL
import tenant_linear_layers_amd as T

A, B, C, D, E, F = (0x1000000 * i for i in range(1, 7))   # never dereferenced


# ------------------------------------------------------------------ C ABI
def test_rms_norm_argument_errors():
    f, g = T.lib().bitdelta_rms_norm, T.lib().bitdelta_rms_norm_mx

    def call(x=A, xs=64, r=B, rs=64, w=C, rows=4, cols=64, h=D, y=E):
        return f(x, xs, r, rs, w, 1e-5, rows, cols, h, y, None)

    def mx(cols=64, y=E, s=F, x=A):
        return g(x, cols, B, cols, C, 1e-5, 4, cols, D, y, s, None)

    assert call(rows=0) == 0 and call(rows=0, x=None, y=None) == 0
    assert call(rows=-1) == 2 and call(cols=0) == 2 and call(rows=1 << 31) == 2
    assert call(rows=1 << 20, cols=1 << 21) == 2 and call(cols=(1 << 30) + 1) == 2
    assert call(xs=-1) == 2 and call(rs=-64) == 2
    assert call(x=None) == 1 and call(w=None) == 1 and call(y=None) == 1
    assert call(r=None) == 1 and call(h=None) == 1          # one without the other
    assert call(x=A + 1) == 3 and call(h=D + 1) == 3 and call(y=E + 1) == 3
    assert call(y=A) == 9 and call(h=B + 8) == 9 and call(y=D + 2) == 9
    assert call(y=A + 2 * 64 * 3, xs=128, rows=3) == 9       # inside a strided x
    assert mx(cols=48) == 2 and mx(s=None) == 1 and mx(y=E + 8) == 3
    assert mx(s=E + 64) == 9 and mx(y=A) == 9


def test_kv_argument_errors():
    w, r = T.lib().bitdelta_kv_write, T.lib().bitdelta_kv_read

    def wr(k=A, v=A + 1024, st=(2048, 128, 2048, 128), slots=B, tokens=3, heads=4, dim=128,
           pages=2, page=16, kc=C, vc=D, ks=None, vs=None):
        return w(k, v, *st, slots, tokens, heads, dim, pages, page, kc, vc, ks, vs, None)

    def rd(slots=B, tokens=3, heads=4, dim=128, pages=2, page=16, kc=C, vc=D, ks=None, vs=None,
           k=E, v=F):
        return r(slots, tokens, heads, dim, pages, page, kc, vc, ks, vs, k, v, None)

    for f in (wr, rd):
        assert f(tokens=0) == 0 and f(tokens=0, slots=None) == 0
        assert f(tokens=-1) == 2 and f(dim=96) == 2 and f(page=8) == 2 and f(page=24) == 2
        assert f(page=65552) == 2 and f(pages=0) == 2 and f(pages=1 << 27) == 2
        assert f(heads=0) == 2 and f(heads=1025) == 2
        assert f(slots=None) == 1 and f(kc=None) == 1 and f(ks=E + 65536) == 1
        assert f(kc=C + 8) == 3 and f(slots=B + 2) == 3
        assert f(kc=D) == 9 or f is rd
    assert wr(st=(-1, 128, 2048, 128)) == 2 and wr(k=A + 1) == 3
    assert wr(kc=A) == 9 and wr(vc=C + 4096) == 9 and wr(ks=C + 16, vs=E) == 9
    assert rd(k=E + 8) == 3 and rd(k=C) == 9 and rd(v=E + 256) == 9 and rd(k=B - 16) == 9


def test_paged_attention_argument_errors():
    f = T.lib().bitdelta_paged_attention

    def call(q=A, st=(1024, 128), kc=B, vc=C, ks=None, vs=None, table=D, cu=D + 4096,
             kv=D + 8192, tokens=5, seqs=2, max_q=4, heads=8, kv_heads=2, dim=128, pages=4,
             page=16, width=3, window=0, out=E, ws=F, wn=1 << 40):
        return f(q, *st, kc, vc, ks, vs, table, cu, kv, tokens, seqs, max_q, heads, kv_heads,
                 dim, pages, page, width, 1.0, window, out, ws, wn, None)

    assert call(tokens=0) == 0 and call(seqs=0) == 0 and call(max_q=0, q=None) == 0
    for bad in (dict(tokens=-1), dict(seqs=-1), dict(seqs=65536), dict(max_q=-1),
                dict(heads=9), dict(heads=0), dict(heads=2048, kv_heads=1024),
                dict(heads=130, kv_heads=2), dict(dim=80), dict(page=20), dict(page=0),
                dict(pages=0), dict(width=-1), dict(width=1 << 28), dict(window=-1),
                dict(tokens=1 << 29), dict(st=(-8, 128)), dict(st=(1024, -1))):
        assert call(**bad) == 2, bad
    for bad in (dict(q=None), dict(kc=None), dict(vc=None), dict(table=None), dict(cu=None),
                dict(kv=None), dict(out=None), dict(ks=F)):
        assert call(**bad) == 1, bad
    for bad in (dict(q=A + 1), dict(kc=B + 8), dict(out=E + 8), dict(table=D + 2),
                dict(cu=D + 4097), dict(kv=D + 2), dict(ws=F + 4), dict(ks=F + 4, vs=F + 65536)):
        assert call(**bad) == 3, bad
    for bad in (dict(out=A), dict(out=B), dict(out=C + 64), dict(out=D)):
        assert call(**bad) == 9, bad
    need = T.paged_attention_workspace_size(5, 2, 4, 8, 2, 128, 3, 16)
    if need:
        assert call(ws=None) == 6 and call(wn=need - 1) == 6 and call(ws=E) == 9
    assert T.paged_attention_workspace_size(5, 2, 4, 9, 2, 128, 3, 16) == 0


def test_paged_attention_refuses_sequences_past_2_to_30_keys():
    """Positions, less a window, have to fit 32 bits."""
    size = T.paged_attention_workspace_size
    assert size(1, 1, 1, 8, 8, 128, 1 << 26, 16) > 0
    assert size(1, 1, 1, 8, 8, 128, (1 << 26) + 1, 16) == 0
    f = T.lib().bitdelta_paged_attention
    assert f(A, 1024, 128, B, C, None, None, D, D + 4096, D + 8192, 1, 1, 1, 8, 8, 128, 4, 16,
             (1 << 26) + 1, 1.0, 0, E, F, 1 << 40, None) == 2


def test_paged_attention_workspace_of_nothing():
    """No sequences, tokens or rows: no workspace, whatever the other sizes."""
    size = T.paged_attention_workspace_size
    for tokens in (0, 1, 5000):
        for seqs in (0, 3):
            for max_q in (0, 1, 5000):
                if tokens and seqs and max_q:
                    continue
                for heads, kv_heads in ((64, 8), (64, 1), (8, 8)):
                    assert size(tokens, seqs, max_q, heads, kv_heads, 128, 300, 16) == 0


@pytest.mark.parametrize("scale", [0.0, -0.125, -0.0, 1e-40, math.inf, -math.inf, math.nan, 3e38])
def test_paged_attention_refuses_scales_that_do_not_keep_the_scores_order(scale):
    f = T.lib().bitdelta_paged_attention
    assert f(A, 1024, 128, B, C, None, None, D, D + 4096, D + 8192, 1, 1, 1, 8, 8, 128, 4, 16, 1,
             scale, 0, E, F, 1 << 40, None) == 2


# ------------------------------------------------------------------ binding
def test_binding_refuses_host_tensors_and_non_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.ones(64, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    c = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16)
    k = x.view(4, 1, 64)
    for call in (lambda: T.rms_norm(x, w, 1e-5), lambda: T.rms_norm_mx(x, w, 1e-5),
                 lambda: T.kv_write(k, k, i, c, c), lambda: T.kv_read(i, c, c),
                 lambda: T.paged_attention(k, c, c, i.view(4, 1), torch.zeros(5), i, 1)):
        with pytest.raises(ValueError, match="device"):
            call()
    with pytest.raises(TypeError):
        T.rms_norm([1.0], w, 1e-5)


# ------------------------------------------------------------------ oracle
def test_oracle_e4m3_matches_torch():
    """The table against torch's e4m3, and the rounding on values between."""
    bits = torch.arange(256, dtype=torch.uint8)
    ours = OL.e4m3_table()
    theirs = bits.view(torch.float8_e4m3fn).float().double().numpy()
    assert np.array_equal(np.isnan(ours), np.isnan(theirs))
    assert np.array_equal(ours[~np.isnan(ours)], theirs[~np.isnan(ours)])
    g = np.random.default_rng(1)
    x = np.concatenate([g.uniform(-448, 448, 4000), g.normal(0, 0.02, 4000),
                        (ours[:126] + ours[1:127]) / 2])       # ties last
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    x32 = torch.from_numpy(x).float().double().numpy()
    assert np.array_equal(OL.e4m3_bits(x32), want)


def test_oracle_scale_borders():
    for e in (-119, -3, 0, 7, 119):
        top = 448.0 * 2.0 ** e
        got = OL.scale_exponent(np.array([top, np.nextafter(top, np.inf), top / 2,
                                          np.nextafter(top / 2, np.inf)]))
        assert list(got) == [e, e + 1, e - 1, e]
    assert list(OL.scale_exponent(np.array([0.0, 1e-300, 2.0 ** 127.9]))) == [-120, -120, 120]


def test_oracle_attention_one_key_and_none():
    g = np.random.default_rng(2)
    k, v = g.normal(size=(3, 1, 16, 64)), g.normal(size=(3, 1, 16, 64))
    q = g.normal(size=(4, 2, 64))
    table = np.array([[2], [1]])
    out, _ = OL.paged_attention(q, k, v, table, [0, 2, 4], [1, 2], window=1)
    assert np.all(out[0] == 0)                              # position -1 sees nothing
    assert np.allclose(out[1], v[2, 0, 0])                  # one key
    assert np.allclose(out[2], v[1, 0, 0]) and np.allclose(out[3], v[1, 0, 1])
    # two equal keys halve the weight; the mean of their values
    k[1, 0, 1] = k[1, 0, 0]
    out, mag = OL.paged_attention(q, k, v, table, [0, 2, 4], [1, 2])
    assert np.allclose(out[3], (v[1, 0, 0] + v[1, 0, 1]) / 2)
    assert np.all(mag >= np.abs(out) - 1e-12) and math.isfinite(mag.sum())
