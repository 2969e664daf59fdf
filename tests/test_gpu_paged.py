"""The paged cache: attention of the newest tokens against the 64-bit definition, and the pages'
operations against the same steps in plain Python, value for value."""
import random

import pytest
import torch

from dynamic_block_sparse_scoring_b200 import abi
from tests.paged_ref import filled
from tests.window_ref import check, visible, window_ref

pytestmark = pytest.mark.gpu

# lens, new, h_q, h_kv, d_qk, d_v, page, window, sink
ATTN = {
    "one_key": ([1], 1, 4, 1, 64, 64, 16, 0, 0),
    "empty_rows": ([0, 5, 0, 0, 33, 0], 1, 8, 2, 128, 128, 16, 0, 0),
    "page_ends": ([15, 16, 17, 63, 64, 65, 127, 128, 129], 1, 16, 4, 128, 128, 64, 0, 0),
    "gqa16_192": ([1000, 1, 517, 64], 1, 64, 4, 192, 128, 64, 0, 0),
    "mha": ([700, 300], 1, 6, 6, 128, 128, 32, 0, 0),
    "group_3": ([250, 31], 1, 6, 2, 64, 128, 128, 0, 0),
    "group_12_64": ([333], 1, 24, 2, 128, 64, 256, 0, 0),
    "group_40": ([333, 90], 1, 40, 1, 128, 128, 16, 0, 0),
    "window": ([900, 64, 65, 1], 1, 8, 2, 128, 128, 16, 64, 0),
    "window_sinks": ([900, 64, 80, 81, 97, 3], 1, 8, 2, 192, 128, 32, 64, 17),
    "window_1": ([900, 2, 1], 1, 8, 2, 64, 64, 64, 1, 0),
    "sinks_cover": ([300, 20], 1, 8, 2, 64, 64, 64, 5, 1000),
    "four_tokens": ([700, 4, 3, 1, 0, 66], 4, 8, 2, 128, 128, 16, 0, 0),
    "four_tokens_window": ([700, 4, 3, 130], 4, 16, 2, 192, 128, 64, 20, 3),
    "nine_tokens_group_7": ([100, 9, 8], 9, 14, 2, 64, 64, 16, 33, 2),
    "d256": ([100, 300], 2, 8, 2, 256, 256, 16, 0, 0),
    "d256_64": ([77], 1, 8, 2, 256, 64, 16, 30, 5),
    "d64_256": ([200, 40], 1, 8, 1, 64, 256, 16, 0, 0),
    "d192_256": ([200, 40], 1, 8, 1, 192, 256, 16, 0, 0),
    "many_rows": ([(37 * i) % 200 for i in range(700)], 1, 4, 2, 64, 64, 16, 0, 0),
    "long": ([40000, 3], 1, 8, 1, 128, 128, 64, 0, 0),
    "long_split_few": ([9001], 1, 2, 2, 64, 64, 128, 0, 0),
}


def make_attn(name, seed=0):
    lens, new, Hq, Hkv, dqk, dv, page, W, ns = ATTN[name]
    cols = -(-max(lens) // page) + 2
    c = filled(len(lens), cols, sum(-(-n // page) for n in lens) + 3, page, Hkv, dqk, dv, lens, seed)
    cfg = abi.paged_config(len(lens), new, Hq, Hkv, dqk, dv, page, len(c.ref), cols, W, ns)
    q = torch.randn(len(lens), new, Hq, dqk, generator=torch.Generator().manual_seed(seed + 1))
    return cfg, c, q.to(torch.bfloat16).cuda()


def check_attn(cfg, c, q, out, lse, what):
    W = cfg.window or 1 << 30
    for b, n in enumerate(c.lens):
        k, v = (x.unsqueeze(0).cuda() for x in c.dense(b))
        if n == 0:
            assert not out[b].any() and torch.isinf(lse[b]).all() and (lse[b] < 0).all(), (what, b)
            continue
        vis = visible(cfg.seqlen_q, n, n - cfg.seqlen_q, W, cfg.sink, "cuda")
        ref = window_ref(q[b:b + 1], k, v, vis, cfg.scale)
        check(out[b:b + 1], ref["out"], f"{what} row {b} out")
        check(lse[b:b + 1], ref["lse"], f"{what} row {b} lse")


@pytest.mark.parametrize("name", sorted(ATTN))
def test_attention(name):
    cfg, c, q = make_attn(name)
    x = c.on_gpu()
    out, lse = abi.paged_attention(cfg, q, x["k_pages"], x["v_pages"], x["table"], x["lens"])
    check_attn(cfg, c, q, out, lse, name)
    again, lse2 = abi.paged_attention(cfg, q, x["k_pages"], x["v_pages"], x["table"], x["lens"])
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    bare = torch.empty_like(out)
    ws = torch.empty(abi.nsa_paged_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    abi.nsa_paged_attn_fwd(cfg, q, x["k_pages"], x["v_pages"], x["table"], x["lens"], bare, None, ws, ws.numel())
    assert torch.equal(out, bare)


def test_ids_and_lengths_out_of_range_stay_in_bounds():
    """The kernel's own checks keep such books from being followed; good rows are not disturbed."""
    cfg, c, q = make_attn("page_ends")
    x = c.on_gpu()
    want, _ = abi.paged_attention(cfg, q, x["k_pages"], x["v_pages"], x["table"], x["lens"])
    x["table"][3, 0], x["table"][6, 1] = 1 << 30, -5
    x["lens"][0], x["lens"][1] = -7, 1 << 30
    out, _ = abi.paged_attention(cfg, q, x["k_pages"], x["v_pages"], x["table"], x["lens"])
    torch.cuda.synchronize()
    good = [2, 4, 5, 7, 8]
    assert torch.equal(out[good], want[good]) and not out[0].any()


# rows, cols, n_pages, page, h_kv, d_qk, d_v
SHAPES = [(5, 9, 40, 16, 2, 64, 64), (7, 6, 30, 64, 1, 192, 128), (3, 20, 50, 32, 3, 128, 256)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("mode", ["wild", "lively"])
def test_a_run_of_page_operations(shape, mode):
    """Appends, forks, shortenings and compactions in random order, every value compared after each.
    The wild run's lists hold mostly entries to be refused; the lively one frees rows more often and
    forks full rows into empty ones."""
    rows, cols, n_pages, page, h, dqk, dv = shape
    rng = random.Random(5)
    lively = mode == "lively"
    c = filled(*shape, lens=[0] * rows, seed=4)
    x = c.on_gpu()
    books = (x["table"], x["lens"], x["ref"])
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    seen = set()
    for step in range(60):
        what = rng.choice(["append", "append", "append", "fork", "free", "keep", "compact"] +
                          (["fork", "fork", "free", "keep"] if lively else []))
        if what == "append":
            most = rng.choice([1, 1, 3, page, 3 * page])
            n_new = [rng.choice([0, 1, most, rng.randint(0, most)]) for _ in range(rows)]
            k_new, v_new = c.new_tokens(rows, most)
            cfg = abi.paged_config(rows, most, h, h, dqk, dv, page, n_pages, cols)
            short = abi.paged_append(cfg, k_new.cuda(), v_new.cuda(), x["k_pages"], x["v_pages"], *books, i32(n_new))
            want = c.append(k_new, v_new, n_new)
            assert int(short) == want, step
            seen.add("short" if want else "appended")
        cfg = abi.paged_config(rows, 1, h, h, dqk, dv, page, n_pages, cols)
        if what == "fork":
            n = rng.randint(1, rows)
            src = [rng.randint(-1, rows) for _ in range(n)]
            dst = [rng.randint(-1, rows) for _ in range(n)]
            if lively:
                full = [b for b in range(rows) if c.lens[b]] or [0]
                dst = [b for b in range(rows) if not c.lens[b]][:n] or [0]
                src = [rng.choice(full) for _ in dst]
            done = abi.pages_fork(cfg, i32(src), i32(dst), *books)
            want = c.fork(src, dst)
            assert done.tolist() == want, step
            seen.update(f"fork{d}" for d in want)
        if what in ("free", "keep"):
            n = rng.randint(1, 2)
            some = [rng.randint(-1, rows) for _ in range(n)]
            keep = None if what == "free" else [rng.randint(-1, cols * page) for _ in range(n)]
            done = abi.pages_free(cfg, i32(some), *books, keep=None if keep is None else i32(keep))
            assert done.tolist() == c.free(some, keep), step
        if what == "compact":
            remap, n_live = abi.pages_compact(cfg, x["k_pages"], x["v_pages"], *books)
            want = c.compact()
            assert (remap.tolist(), int(n_live)) == want, step
        c.assert_equal(x, f"step {step} {what}")
    assert {"appended", "fork1" if lively else "fork0"} <= seen, seen


def test_sharers_of_one_last_page():
    """Three rows hold a page that is not full: all append, then some."""
    for n_new, copies in [([1, 1, 1, 0], 2), ([1, 0, 2, 0], 2), ([0, 1, 0, 0], 1)]:
        c = filled(4, 4, 20, 16, 2, 64, 64, [21, 0, 0, 5], seed=9)
        x = c.on_gpu()
        books = (x["table"], x["lens"], x["ref"])
        cfg = abi.paged_config(4, 2, 2, 2, 64, 64, 16, 20, 4)
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        abi.pages_fork(cfg, i32([0, 0]), i32([1, 2]), *books)
        c.fork([0, 0], [1, 2])
        k_new, v_new = c.new_tokens(4, 2)
        used = sum(r > 0 for r in c.ref)
        assert int(abi.paged_append(cfg, k_new.cuda(), v_new.cuda(), x["k_pages"], x["v_pages"], *books,
                                    i32(n_new))) == 0
        assert c.append(k_new, v_new, n_new) == 0
        c.assert_equal(x, str(n_new))
        assert sum(r > 0 for r in c.ref) == used + copies


@pytest.mark.parametrize("page", [16, 256])
@pytest.mark.parametrize("keeper", [2, 0])
def test_sharers_with_different_lengths_on_one_page(page, keeper):
    """Rows share their last page with different lengths (some were shortened): the row that keeps
    it, the last one, writes over what the others still copy.  Row 3 has another page, shared with 4."""
    rows = 40
    rng = random.Random(6)
    c = filled(rows, 4, 4 * rows, page, 3, 192, 128, [2 * page - 1, 0, 0, page - 3, 0], seed=10)
    x = c.on_gpu()
    books = (x["table"], x["lens"], x["ref"])
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    cfg = abi.paged_config(rows, 1, 3, 3, 192, 128, page, 4 * rows, 4)
    src, dst = [0] * (rows - 3) + [3], [b for b in range(1, rows) if b not in (3, 4)] + [4]
    assert abi.pages_fork(cfg, i32(src), i32(dst), *books).tolist() == c.fork(src, dst)
    some = [b for b in range(rows) if b not in (3, rows - 1)] + [rows - 1]
    keep = [page + rng.randint(1, page - 1) if b != 4 else rng.randint(1, page - 4) for b in some[:-1]]
    keep.append(page + 1 + keeper)
    assert abi.pages_free(cfg, i32(some), *books, keep=i32(keep)).tolist() == c.free(some, keep)
    cfg = abi.paged_config(rows, page, 3, 3, 192, 128, page, 4 * rows, 4)
    k_new, v_new = c.new_tokens(rows, page)
    assert int(abi.paged_append(cfg, k_new.cuda(), v_new.cuda(), x["k_pages"], x["v_pages"], *books)) == 0
    assert c.append(k_new, v_new, [page] * rows) == 0
    c.assert_equal(x)


def test_n_new_null_appends_everything_and_a_full_pool_changes_nothing():
    c = filled(3, 8, 9, 16, 2, 128, 64, [20, 0, 16], seed=2)
    x = c.on_gpu()
    books = (x["table"], x["lens"], x["ref"])
    cfg = abi.paged_config(3, 12, 2, 2, 128, 64, 16, 9, 8)
    for _ in range(4):
        k_new, v_new = c.new_tokens(3, 12)
        short = abi.paged_append(cfg, k_new.cuda(), v_new.cuda(), x["k_pages"], x["v_pages"], *books)
        assert int(short) == c.append(k_new, v_new, [12] * 3)
        c.assert_equal(x)
    assert int(short) > 0
    cfg = abi.paged_config(3, 12, 2, 2, 128, 64, 16, 9, 3)       # a table of three columns
    narrow = [books[0][:, :3].contiguous(), books[1], books[2]]
    before = [t.clone() for t in narrow]
    assert int(abi.paged_append(cfg, k_new.cuda(), v_new.cuda(), x["k_pages"], x["v_pages"], *narrow)) == -1
    assert all(torch.equal(a, b) for a, b in zip(before, narrow))


def test_prompt_then_decode_then_fork_then_compact():
    """The operators as they are used together: a prompt's attention over contiguous K/V, the prompt
    put into pages, tokens decoded from them, a fork that decodes on its own, and a compaction that
    changes no output; every decoded row is the row that the prompt form gives."""
    Hq, Hkv, dqk, dv, page, W, ns = 16, 2, 128, 128, 16, 40, 5
    T, P0 = 75, 60
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, k, v = r(2, T, Hq, dqk), r(2, Hkv, T, dqk), r(2, Hkv, T, dv)
    whole, _ = abi.window_forward(abi.window_config(2, T, T, Hq, Hkv, dqk, dv, W, ns), q, k, v)
    ref = window_ref(q, k, v, visible(T, T, 0, W, ns, "cuda"), dqk ** -0.5)["out"]
    check(whole, ref, "prompt")
    rows, cols, n_pages = 4, 8, 40
    kp = torch.full((n_pages, Hkv, page, dqk), float("nan"), dtype=torch.bfloat16, device="cuda")
    vp = torch.full((n_pages, Hkv, page, dv), float("nan"), dtype=torch.bfloat16, device="cuda")
    table = torch.full((rows, cols), -1, dtype=torch.int32, device="cuda")
    lens, ref_n = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (rows, n_pages))
    pad = lambda x: torch.cat([x, torch.zeros_like(x)]).contiguous()  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731

    def put(t0, t1, n_new):
        cfg = abi.paged_config(rows, t1 - t0, Hq, Hkv, dqk, dv, page, n_pages, cols, W, ns)
        assert int(abi.paged_append(cfg, pad(k[:, :, t0:t1]), pad(v[:, :, t0:t1]), kp, vp, table, lens, ref_n,
                                    i32(n_new))) == 0

    put(0, P0, [P0, P0, 0, 0])
    cfg = abi.paged_config(rows, 1, Hq, Hkv, dqk, dv, page, n_pages, cols, W, ns)
    assert abi.pages_fork(cfg, i32([0, 1]), i32([2, 3]), table, lens, ref_n).tolist() == [1, 1]
    twice = lambda x: torch.cat([x, x]).contiguous()  # noqa: E731
    for t in range(P0, T):
        c1 = abi.paged_config(rows, 1, Hq, Hkv, dqk, dv, page, n_pages, cols, W, ns)
        assert int(abi.paged_append(c1, twice(k[:, :, t:t + 1]), twice(v[:, :, t:t + 1]), kp, vp, table, lens,
                                    ref_n)) == 0
        out, _ = abi.paged_attention(cfg, twice(q[:, t:t + 1]), kp, vp, table, lens)
        assert torch.equal(out[:2], out[2:])
        check(out[:2], (ref[0][:, t:t + 1], ref[1][:, t:t + 1]), f"token {t}")
        if t == P0 + 5:
            abi.pages_free(cfg, i32([0]), table, lens, ref_n)
            abi.pages_compact(cfg, kp, vp, table, lens, ref_n)
            moved, _ = abi.paged_attention(cfg, twice(q[:, t:t + 1]), kp, vp, table, lens)
            # the shares follow the lengths, so a row's sum is cut elsewhere once another row is
            # empty: the same values within the bound, not the same bits
            check(moved[2:], (ref[0][:, t:t + 1], ref[1][:, t:t + 1]), "after the compaction")
            assert not moved[0].any()
            perm = torch.randperm(n_pages, generator=torch.Generator().manual_seed(1)).cuda()
            other = torch.where(table >= 0, perm[table.clamp(min=0).long()].to(torch.int32), table)
            kq, vq = torch.empty_like(kp), torch.empty_like(vp)
            kq[perm], vq[perm] = kp, vp
            placed, _ = abi.paged_attention(cfg, twice(q[:, t:t + 1]), kq, vq, other, lens)
            assert torch.equal(placed, moved)          # the pages' places change no bit
            assert abi.pages_fork(cfg, i32([2]), i32([0]), table, lens, ref_n).tolist() == [1]
    assert torch.equal((table >= 0).sum(1).cpu(), torch.tensor([5, 5, 5, 5]))


def test_a_captured_step_serves_a_growing_cache():
    """Append and attention of one token in one graph, replayed while the rows grow over page ends."""
    c = filled(3, 8, 24, 16, 2, 128, 128, [14, 30, 0], seed=3)
    x = c.on_gpu()
    books = (x["table"], x["lens"], x["ref"])
    cfg = abi.paged_config(3, 1, 8, 2, 128, 128, 16, 24, 8)
    k_new, v_new = (t.cuda() for t in c.new_tokens(3, 1))
    q = torch.zeros(3, 1, 8, 128, dtype=torch.bfloat16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    saved = {n: t.clone() for n, t in x.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                                   # warm-up
        abi.paged_append(cfg, k_new, v_new, x["k_pages"], x["v_pages"], *books)
        abi.paged_attention(cfg, q, x["k_pages"], x["v_pages"], x["table"], x["lens"])
    torch.cuda.current_stream().wait_stream(side)
    for n in x:
        x[n].copy_(saved[n])
    with torch.cuda.graph(graph):
        short = abi.paged_append(cfg, k_new, v_new, x["k_pages"], x["v_pages"], *books)
        out, lse = abi.paged_attention(cfg, q, x["k_pages"], x["v_pages"], x["table"], x["lens"])
    for step in range(6):
        kn, vn = c.new_tokens(3, 1)
        k_new.copy_(kn)
        v_new.copy_(vn)
        q.copy_(torch.randn(q.shape, generator=c.g).to(torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        assert int(short) == 0 and c.append(kn, vn, [1, 1, 1]) == 0
        c.assert_equal(x, f"step {step}")
        check_attn(cfg, c, q, out, lse, f"step {step}")


def test_offsets_past_32_bits():
    """A pool of more than 2^31 elements whose last pages are in use: attention, append, compaction."""
    n_pages, page, h, d = 70000, 64, 4, 128
    c = filled(2, 6, 12, page, h, d, d, [200, 130], seed=6)
    x = c.on_gpu()
    kp = torch.full((n_pages, h, page, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    vp = torch.full((n_pages, h, page, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    assert kp.numel() > 1 << 31
    off = n_pages - 12
    kp[off:], vp[off:] = x["k_pages"], x["v_pages"]
    table = torch.where(x["table"] >= 0, x["table"] + off, x["table"])
    ref = torch.ones(n_pages, dtype=torch.int32, device="cuda")        # the others are held elsewhere
    ref[off:] = x["ref"]
    lens = x["lens"].clone()
    cfg = abi.paged_config(2, 1, 8, h, d, d, page, n_pages, 6)
    q = torch.randn(2, 1, 8, d, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).cuda()
    out, lse = abi.paged_attention(cfg, q, kp, vp, table, lens)
    check_attn(cfg, c, q, out, lse, "far pages")
    k_new, v_new = c.new_tokens(2, 70)
    grow = abi.paged_config(2, 70, 8, h, d, d, page, n_pages, 6)
    assert int(abi.paged_append(grow, k_new.cuda(), v_new.cuda(), kp, vp, table, lens, ref)) == 0
    assert c.append(k_new, v_new, [70, 70]) == 0
    ref[:off] = 0                                                      # now the pool's beginning is free
    remap, n_live = abi.pages_compact(cfg, kp, vp, table, lens, ref)
    assert int(n_live) == sum(n > 0 for n in c.ref) and int(table.max()) < int(n_live)
    out, lse = abi.paged_attention(cfg, q, kp, vp, table, lens)
    check_attn(cfg, c, q, out, lse, "after the compaction")


def test_two_streams_with_workspaces_of_their_own():
    """Calls that overlap on two streams, each with its own outputs and workspace."""
    made = [make_attn(n, seed=7) for n in ("gqa16_192", "window_sinks")]
    xs = [c.on_gpu() for _, c, _ in made]
    want = [abi.paged_attention(cfg, q, x["k_pages"], x["v_pages"], x["table"], x["lens"])
            for (cfg, _, q), x in zip(made, xs)]
    streams = [torch.cuda.Stream() for _ in made]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, ((cfg, _, q), x) in enumerate(zip(made, xs)):
            with torch.cuda.stream(streams[i]):
                got[i].append(abi.paged_attention(cfg, q, x["k_pages"], x["v_pages"], x["table"], x["lens"]))
    torch.cuda.synchronize()
    for w, many in zip(want, got):
        for o, l in many:
            assert torch.equal(o, w[0]) and torch.equal(l, w[1])


@pytest.mark.parametrize("lens, h_q", [([40, 7], 8), ([5000, 7], 8), ([5000, 7], 2)])
def test_a_key_that_is_not_a_number_shows_in_out_and_lse(lens, h_q):
    """One NaN among a row's keys, in a unit that one warp finishes and in one that is cut and joined:
    the row's out and lse are NaN (not -inf, which stands for no key), the other rows' are as before."""
    c = filled(2, 80, 90, 64, 2, 128, 128, lens, seed=12)
    cfg = abi.paged_config(2, 1, h_q, 2, 128, 128, 64, 90, 80)
    q = torch.randn(2, 1, h_q, 128, generator=torch.Generator().manual_seed(13)).to(torch.bfloat16).cuda()
    x = c.on_gpu()
    want = abi.paged_attention(cfg, q, x["k_pages"], x["v_pages"], x["table"], x["lens"])
    x["k_pages"][c.table[0][0], 0, 3, 5] = float("nan")              # KV head 0 of row 0
    out, lse = abi.paged_attention(cfg, q, x["k_pages"], x["v_pages"], x["table"], x["lens"])
    G = h_q // 2
    assert out[0, :, :G].isnan().all() and lse[0, :, :G].isnan().all()
    assert torch.equal(out[0, :, G:], want[0][0, :, G:]) and torch.equal(lse[0, :, G:], want[1][0, :, G:])
    assert torch.equal(out[1], want[0][1]) and torch.equal(lse[1], want[1][1])
