"""Refusals of the decoder-layer operators at their limits, without a GPU: each
call below is refused on the host before anything is enqueued."""

import tenant_linear_layers_amd as T

A, B, C, D, E, F = (0x1000000 * i for i in range(1, 7))   # never dereferenced


def test_one_alignment_for_a_cache_and_its_scales():
    """A cache that can be written can be read and attended over."""
    L = T.lib()

    def write(ks, vs):
        return L.bitdelta_kv_write(A, A + 1024, 2048, 128, 2048, 128, B, 3, 4, 128, 2, 16, C, D,
                                   ks, vs, None)

    def read(ks, vs):
        return L.bitdelta_kv_read(B, 3, 4, 128, 2, 16, C, D, ks, vs, A, A + 65536, None)

    def attend(ks, vs):
        return L.bitdelta_paged_attention(A, 1024, 128, C, D, ks, vs, B, B + 4096, B + 8192, 5, 2,
                                          4, 8, 4, 128, 2, 16, 1, 1.0, 0, A + 65536, None, 0,
                                          None)

    for call in (write, read, attend):
        for off in (1, 2, 4, 8):
            assert call(E + off, F) == 3 and call(E, F + off) == 3, (call.__name__, off)


def test_attention_refuses_a_workspace_that_is_missing_small_or_the_output():
    """Sequences long enough to be cut: of few rows, of many, and of both."""
    f = T.lib().bitdelta_paged_attention

    def call(tokens, seqs, max_q, ws, wn, out=F):
        return f(A, 1024, 128, C, D, None, None, B, B + 65536, B + 131072, tokens, seqs, max_q, 8,
                 2, 128, 64, 16, 64, 1.0, 0, out, ws, wn, None)

    for sizes in ((2, 2, 1), (40, 1, 40), (45, 6, 40)):
        need = T.paged_attention_workspace_size(*sizes, 8, 2, 128, 64, 16)
        assert need > 0
        assert call(*sizes, None, 0) == 6 and call(*sizes, None, need) == 6
        assert call(*sizes, E, need - 1) == 6 and call(*sizes, E, 0) == 6
        assert call(*sizes, E + 8, need) == 3
        assert call(*sizes, F, need) == 9 and call(*sizes, F - need + 16, need) == 9
        assert call(*sizes, A, need) == 9 and call(*sizes, C, need) == 9
