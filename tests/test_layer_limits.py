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
