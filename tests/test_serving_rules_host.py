"""The serving calls' rules that need no GPU: what a workspace is sized for, and soft caps
that fp32 cannot work with."""

import math

import pytest

import block_sparse_attention_48_b200 as fa


@pytest.mark.parametrize("shape", [
    # B, Hq, Hkv, q_len, D: shapes that the calls refuse
    (1, 8, 1, 1024, 64), (1, 4096, 1, 1, 64), (2, 34, 2, 1, 128), (2, 8, 2, 5, 64), (2, 8, 3, 1, 64), (2, 8, 2, 1, 96),
    (2, 8, 2, 1, 10 ** 6), (65536, 8, 2, 1, 64), (1, 65536, 65536, 1, 64), (1, 1, 1, 2 ** 62, 64),
    (1, 2 ** 62, 1, 4, 64), (2 ** 40, 0, 1, 1, 64), (-1, 8, 2, 1, 64), (1, 8, 2, -1, 64)])
def test_no_workspace_for_refused_shapes(shape):
    lib = fa.library()
    assert lib.fa_decode_paged_workspace_size(*shape) == 0
    for prefix in (0, 128, 2 ** 31 - 256):
        assert lib.fa_decode_shared_workspace_size(*shape, prefix) == 0


def test_workspaces_of_taken_shapes():
    lib = fa.library()
    for B, Hq, Hkv, n, D in ((1, 16, 1, 1, 64), (65535, 4, 4, 1, 128), (3, 12, 4, 5, 64)):
        paged = lib.fa_decode_paged_workspace_size(B, Hq, Hkv, n, D)
        assert paged > 256 and lib.fa_decode_shared_workspace_size(B, Hq, Hkv, n, D, 0) == paged
    # nothing to do: the status word
    for B, Hq, n in ((0, 8, 1), (2, 0, 1), (2, 64, 0)):
        assert lib.fa_decode_paged_workspace_size(B, Hq, 2, n, 64) == 256
        assert lib.fa_decode_shared_workspace_size(B, Hq, 2, n, 64, 2 ** 31 - 256) == 256
    # a prefix's work list of 2^31 entries is refused
    assert lib.fa_decode_shared_workspace_size(65535, 16, 1, 1, 64, 2 ** 31 - 256) == 0


@pytest.mark.parametrize("shared", [False, True])
def test_soft_caps_beyond_fp32_are_refused(shared):
    """The kernels multiply by scale / cap and by cap log2(e): both must be finite, or every
    output would be NaN."""
    lib = fa.library()

    def tensor(dims, data=4096):
        t = fa.TensorDesc()
        t.data = data
        for i in range(4):
            t.dims[i], t.strides[i] = dims[i], math.prod(dims[i + 1:])
        return t
    q, pool = tensor([2, 8, 1, 64]), tensor([5, 2, 128, 64])
    sm = fa.ScoreModDesc()
    sm.kind = fa.SCORE["softcap"]

    def call(cap, scale):
        sm.softcap = cap
        fn = lib.fa_decode_shared if shared else lib.fa_decode_paged
        return fn(q, pool, pool, 4096, 3, 3, 4096, 128 if shared else -1, sm, scale, q, None, 4096, 1 << 30, None)
    for cap, scale in ((math.inf, 0.0), (math.nan, 0.0), (3e38, 0.0), (1e-40, 0.0), (1e-30, 1e10), (-1.0, 0.0)):
        assert call(cap, scale) == fa.FA_ERR_INVALID_ARG
