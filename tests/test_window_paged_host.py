"""Host-side checks of the window attention's and the paged cache's entry points: bad arguments are
refused before anything is launched (the addresses below are never followed)."""
import ctypes

import pytest

P = 1 << 20                     # an aligned address that nothing reads


@pytest.fixture(scope="module")
def abi():
    from dynamic_block_sparse_scoring_b200 import build
    build.build()
    from dynamic_block_sparse_scoring_b200 import abi as a
    return a


def _status(abi, f):
    with pytest.raises(abi.NsaError) as e:
        f()
    return abi.STATUS[e.value.status]


def _win(abi, **kw):
    f = dict(batch=2, seqlen_q=64, seqlen_kv=96, h_q=8, h_kv=2, d_qk=128, d_v=128, window=32, sink=4, q_pos0=32)
    f.update(kw)
    return abi.window_config(**f)


def _paged(abi, **kw):
    f = dict(batch=2, seqlen_q=1, h_q=8, h_kv=2, d_qk=128, d_v=128, page_size=64, n_pages=10, max_pages=4)
    f.update(kw)
    return abi.paged_config(**f)


def test_struct_layouts_match_the_header(abi):
    assert ctypes.sizeof(abi.NsaWindowConfig) == 12 * 4 and ctypes.sizeof(abi.NsaPagedConfig) == 13 * 4


WIN_BAD = [dict(batch=0), dict(seqlen_q=-1), dict(seqlen_kv=0), dict(q_pos0=-1), dict(q_pos0=33), dict(h_q=7),
           dict(h_q=0), dict(h_kv=0), dict(d_qk=0), dict(d_v=-1), dict(window=0), dict(window=-5), dict(sink=-1),
           dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=1e-31), dict(scale=1e31)]
WIN_OFF = [dict(d_qk=96), dict(d_qk=320), dict(d_v=192), dict(d_v=32),
           dict(seqlen_q=1, seqlen_kv=2 ** 31 - 1, q_pos0=0), dict(batch=1 << 20, seqlen_q=1 << 12, seqlen_kv=1 << 12,
                                                                   q_pos0=0)]


@pytest.mark.parametrize("kw", WIN_BAD + WIN_OFF, ids=str)
def test_window_configs_are_refused(abi, kw):
    want = "NSA_ERR_INVALID_ARG" if kw in WIN_BAD else "NSA_ERR_UNSUPPORTED"
    cfg = _win(abi, **kw)
    assert _status(abi, lambda: abi.nsa_window_attn_fwd(cfg, P, P, P, P, P)) == want
    assert _status(abi, lambda: abi.nsa_window_attn_bwd(cfg, P, P, P, P, P, P, P, P, P, P, 1 << 40)) == want
    assert _status(abi, lambda: abi.nsa_window_bwd_workspace_size(cfg)) == want


def test_window_flags_and_null_config(abi):
    cfg = _win(abi)
    cfg.flags = 1
    assert _status(abi, lambda: abi.nsa_window_attn_fwd(cfg, P, P, P, P, P)) == "NSA_ERR_INVALID_ARG"
    assert abi.lib.nsa_window_attn_fwd(None, P, P, P, P, P, None) == 1


@pytest.mark.parametrize("bad", [None, P + 2])
def test_window_pointers(abi, bad):
    cfg = _win(abi)
    ws = abi.nsa_window_bwd_workspace_size(cfg)
    for i in range(5):
        if bad is None and i == 4:
            continue                                     # lse may be NULL
        args = [P] * 5
        args[i] = bad
        assert _status(abi, lambda: abi.nsa_window_attn_fwd(cfg, *args)) == "NSA_ERR_INVALID_ARG"
    for i in range(9):
        args = [P] * 9
        args[i] = bad
        assert _status(abi, lambda: abi.nsa_window_attn_bwd(cfg, *args, P, ws)) == "NSA_ERR_INVALID_ARG"
    assert _status(abi, lambda: abi.nsa_window_attn_bwd(cfg, *[P] * 9, P, ws - 1)) == "NSA_ERR_WORKSPACE"
    assert _status(abi, lambda: abi.nsa_window_attn_bwd(cfg, *[P] * 9, None, ws)) == "NSA_ERR_WORKSPACE"


def test_zero_queries_need_no_query_buffers(abi):
    cfg = _win(abi, seqlen_q=0)
    abi.nsa_window_attn_fwd(cfg, None, P, P, None)
    assert _status(abi, lambda: abi.nsa_window_attn_fwd(cfg, None, None, P, None)) == "NSA_ERR_INVALID_ARG"
    assert _status(abi, lambda: abi.nsa_window_attn_bwd(cfg, None, P, P, None, None, None, None, None, P)) \
        == "NSA_ERR_INVALID_ARG"


PAGED_BAD = [dict(batch=0), dict(seqlen_q=0), dict(n_pages=0), dict(max_pages=0), dict(h_q=7), dict(h_kv=0),
             dict(d_qk=0), dict(d_v=0), dict(page_size=0), dict(window=-1), dict(sink=-1), dict(scale=0.0),
             dict(scale=float("nan"))]
PAGED_OFF = [dict(d_qk=96), dict(d_v=192), dict(page_size=8), dict(page_size=48), dict(page_size=512),
             dict(max_pages=1 << 25), dict(batch=1 << 20, max_pages=1 << 12)]


@pytest.mark.parametrize("kw", PAGED_BAD + PAGED_OFF, ids=str)
def test_paged_configs_are_refused(abi, kw):
    want = "NSA_ERR_INVALID_ARG" if kw in PAGED_BAD else "NSA_ERR_UNSUPPORTED"
    cfg = _paged(abi, **kw)
    big = 1 << 40
    for f in [lambda: abi.nsa_paged_attn_fwd(cfg, P, P, P, P, P, P, P, P, big),
              lambda: abi.nsa_paged_append(cfg, P, P, P, P, P, P, P, P, P, P, big),
              lambda: abi.nsa_pages_fork(cfg, 1, P, P, P, P, P, P),
              lambda: abi.nsa_pages_free(cfg, 1, P, P, P, P, P, P),
              lambda: abi.nsa_pages_compact(cfg, P, P, P, P, P, P, P, P, big),
              lambda: abi.nsa_paged_workspace_size(cfg), lambda: abi.nsa_paged_append_workspace_size(cfg),
              lambda: abi.nsa_pages_compact_workspace_size(cfg)]:
        assert _status(abi, f) == want


def test_paged_limits(abi):
    assert _status(abi, lambda: abi.nsa_paged_append(_paged(abi, batch=8193), P, P, P, P, P, P, P, P, P, P, 1 << 40)) \
        == "NSA_ERR_UNSUPPORTED"
    assert _status(abi, lambda: abi.nsa_pages_fork(_paged(abi), -1, P, P, P, P, P, P)) == "NSA_ERR_INVALID_ARG"
    assert _status(abi, lambda: abi.nsa_pages_free(_paged(abi), -1, P, P, P, P, P, P)) == "NSA_ERR_INVALID_ARG"
    abi.nsa_pages_fork(_paged(abi), 0, None, None, P, P, P, None)      # nothing to do
    abi.nsa_pages_free(_paged(abi), 0, None, None, P, P, P, None)


@pytest.mark.parametrize("bad", [None, P + 4])
def test_paged_pointers(abi, bad):
    cfg = _paged(abi)
    n = abi.nsa_paged_workspace_size(cfg)
    for i in range(7):
        if bad is None and i == 6:
            continue                                     # lse may be NULL
        args = [P] * 7
        args[i] = bad
        assert _status(abi, lambda: abi.nsa_paged_attn_fwd(cfg, *args, P, n)) == "NSA_ERR_INVALID_ARG"
    assert _status(abi, lambda: abi.nsa_paged_attn_fwd(cfg, *[P] * 7, P, n - 1)) == "NSA_ERR_WORKSPACE"
    n = abi.nsa_paged_append_workspace_size(cfg)
    for i in range(9):
        if (bad is None and i == 2) or (bad is not None and i == 8):
            continue                                     # n_new may be NULL; short_pages needs 4 bytes only
        args = [P] * 9
        args[i] = bad
        assert _status(abi, lambda: abi.nsa_paged_append(cfg, *args, P, n)) == "NSA_ERR_INVALID_ARG"
    assert _status(abi, lambda: abi.nsa_paged_append(cfg, *[P] * 9, P, n - 1)) == "NSA_ERR_WORKSPACE"
    n = abi.nsa_pages_compact_workspace_size(cfg)
    for i in range(7):
        if bad is not None and i == 6:
            continue                                     # n_live needs 4 bytes only
        args = [P] * 7
        args[i] = bad
        assert _status(abi, lambda: abi.nsa_pages_compact(cfg, *args, P, n)) == "NSA_ERR_INVALID_ARG"
    assert _status(abi, lambda: abi.nsa_pages_compact(cfg, *[P] * 7, P, n - 1)) == "NSA_ERR_WORKSPACE"
    for i in range(6):
        args = [P] * 6
        args[i] = None
        if i != 5:
            assert _status(abi, lambda: abi.nsa_pages_fork(cfg, 1, *args)) == "NSA_ERR_INVALID_ARG"
        if i not in (1, 5):
            assert _status(abi, lambda: abi.nsa_pages_free(cfg, 1, *args)) == "NSA_ERR_INVALID_ARG"


def test_wrappers_refuse_host_tensors(abi):
    import torch
    q = torch.zeros(2, 64, 8, 128, dtype=torch.bfloat16)
    k = torch.zeros(2, 2, 96, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        abi.window_forward(_win(abi), q, k, k)


def test_waits_for_tensor_memory_name_the_registers():
    """A load from tensor memory is asynchronous, and only a wait that names its registers keeps the
    compiler from moving their uses before it: the window kernels use no other."""
    import pathlib

    import dynamic_block_sparse_scoring_b200 as pkg
    for src in pathlib.Path(pkg.__file__).parent.joinpath("csrc").glob("window_*.cu"):
        text = src.read_text()
        assert "tmem_wait_ld()" not in text, src.name
        assert "tmem_ld32(" not in text or "tmem_wait_ld32(" in text, src.name


def test_fork_and_free_refuse_misaligned_books_and_lists(abi):
    """The cache's books are 16-byte aligned as in every other call on it; lists, and the single results
    of append and compaction, hold whole int32."""
    cfg = _paged(abi)
    for f, lists in [(abi.nsa_pages_fork, (0, 1, 5)), (abi.nsa_pages_free, (0, 1, 5))]:
        for i in range(6):
            args = [P] * 6
            args[i] = P + (2 if i in lists else 4)
            assert _status(abi, lambda: f(cfg, 1, *args)) == "NSA_ERR_INVALID_ARG", (f.__name__, i)
        args = [P] * 6
        args[3] = P + 4
        assert _status(abi, lambda: f(cfg, 0, *args)) == "NSA_ERR_INVALID_ARG"
    n = abi.nsa_paged_append_workspace_size(cfg)
    assert _status(abi, lambda: abi.nsa_paged_append(cfg, *[P] * 8, P + 2, P, n)) == "NSA_ERR_INVALID_ARG"
    n = abi.nsa_pages_compact_workspace_size(cfg)
    assert _status(abi, lambda: abi.nsa_pages_compact(cfg, *[P] * 6, P + 2, P, n)) == "NSA_ERR_INVALID_ARG"


def test_sizes_whose_products_pass_64_bits_are_refused(abi):
    """2^22 sequences of 2^21 tokens and heads: the product is 2^64, which must not count as 0."""
    big = dict(batch=1 << 22, seqlen_q=1 << 21, seqlen_kv=1 << 21, h_q=1 << 21, h_kv=1 << 21, q_pos0=0)
    for kw in [big, dict(big, seqlen_q=0), dict(big, batch=1 << 30, h_q=1 << 30, h_kv=1 << 30, seqlen_kv=16, seqlen_q=16)]:
        cfg = _win(abi, **kw)
        assert _status(abi, lambda: abi.nsa_window_bwd_workspace_size(cfg)) == "NSA_ERR_UNSUPPORTED"
        assert _status(abi, lambda: abi.nsa_window_attn_fwd(cfg, P, P, P, P, P)) == "NSA_ERR_UNSUPPORTED"
    cfg = _paged(abi, batch=1 << 30, max_pages=1, h_q=1 << 28, h_kv=1 << 14, seqlen_q=1 << 10)
    assert (1 << 30) * (1 << 14) * (1 << 20) == 1 << 64          # sequences, KV heads, tiles of 16 rows
    assert _status(abi, lambda: abi.nsa_paged_attn_fwd(cfg, *[P] * 7, P, 1 << 40)) == "NSA_ERR_UNSUPPORTED"


@pytest.mark.parametrize("big", [1 << 31, (1 << 32) + 5, 1 << 40])
def test_configs_refuse_counts_that_do_not_fit(abi, big):
    """No count is taken modulo 2^32; a window or a number of sinks that large covers every key."""
    for kw in [dict(seqlen_kv=big), dict(batch=big)]:
        with pytest.raises(ValueError, match="31 bits"):
            _win(abi, **kw)
    for kw in [dict(n_pages=big), dict(page_size=big)]:
        with pytest.raises(ValueError, match="31 bits"):
            _paged(abi, **kw)
    for make in (_win, _paged):
        cfg = make(abi, window=big, sink=big)
        assert cfg.window == cfg.sink == 2 ** 31 - 1
