"""Page tables, slot maps and block tables on the GPU, against a plain scheduler
(tests/draw_util.py), and a whole decode step: pages, verification, history and
the pages of refused drafts back."""
import numpy as np
import pytest

import token_sampling_logits_gb300 as gs
from tests import draw_util as du

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def dev(a, dtype):
    return torch.tensor(np.asarray(a), dtype=dtype, device="cuda")


def offsets_of(counts):
    return dev(np.concatenate([[0], np.cumsum(counts)]), torch.int64)


def check_state(st, ref):
    assert np.array_equal(st.table.cpu().numpy(), ref.table())
    assert st.length.tolist() == ref.length
    assert st.free_count.tolist() == [len(ref.free)]
    assert st.free.tolist()[:len(ref.free)] == ref.free


def step(st, ref, counts, slots, columns, named=True):
    n, total = len(counts), int(np.sum(counts))
    table = torch.full((n, columns + 2), -9, dtype=torch.int32, device="cuda")
    lengths = torch.empty(n, dtype=torch.int32, device="cuda")
    maps = torch.full((total + 2,), -9, dtype=torch.int64, device="cuda")
    one = all(c == 1 for c in counts)
    start, _ = gs.pages_extend(st, total, slots=dev(slots, torch.int32) if named else None,
                               offsets=None if one else offsets_of(counts),
                               slot_map=maps[1:1 + total], lengths=lengths, table=table[:, :columns])
    rs, rm, rl, rt = ref.extend(counts, slots)
    assert start.tolist() == rs
    assert maps.tolist() == [-9] + sum(rm, []) + [-9]
    assert lengths.tolist() == rl
    want = np.array([(t + [-1] * columns)[:columns] for t in rt], np.int32).reshape(n, columns)
    assert np.array_equal(table[:, :columns].cpu().numpy(), want)
    assert (table[:, columns:] == -9).all()
    check_state(st, ref)
    return start, rs


@pytest.mark.parametrize("slots,pages,page,columns", [
    (1, 1, 1, 1), (5, 40, 4, 9), (64, 500, 16, 20), (300, 900, 7, 30), (2500, 9000, 3, 12)])
@pytest.mark.parametrize("seed", [0, 1])
def test_extend_and_trim(slots, pages, page, columns, seed):
    rng = np.random.default_rng(slots + seed)
    st, ref = gs.new_page_state(slots, pages, page, columns), du.Pages(slots, pages, page, columns)
    check_state(st, ref)
    for turn in range(8):
        n = int(rng.integers(1, slots + 1))
        which = rng.permutation(slots)[:n]
        if turn == 3:  # slots out of range or named twice
            which = rng.integers(-2, slots + 2, n)
        counts = rng.integers(0, [2, 3 * page, columns * page][turn % 3] + 1, n)
        if turn == 1:
            counts[:] = 1
        cols = int(rng.integers(0, columns + 3))
        start, rs = step(st, ref, counts, which.tolist(), cols)
        keep = rng.integers(-1, counts.max() + 2, n)
        if turn % 2:
            gs.pages_trim(st, slots=dev(which, torch.int32), start=start, keep=dev(keep, torch.int32))
            ref.trim(which.tolist(), rs, keep.tolist())
        elif turn == 6:
            gs.pages_trim(st, slots=dev(which, torch.int32))
            ref.trim(which.tolist(), [0] * n, [0] * n)
        check_state(st, ref)
    gs.pages_trim(st)
    ref.trim(range(slots), [0] * slots, [0] * slots)
    check_state(st, ref)
    assert st.free_count.item() == pages and sorted(st.free.tolist()) == list(range(pages))


def test_a_step_taken_back_leaves_the_state_as_it_was():
    rng = np.random.default_rng(3)
    st, ref = gs.new_page_state(50, 400, 8, 16), du.Pages(50, 400, 8, 16)
    step(st, ref, rng.integers(0, 60, 50), rng.permutation(50).tolist(), 16)
    before = [t.clone() for t in (st.table, st.length, st.free, st.free_count)]
    which = dev(rng.permutation(50)[:30], torch.int32)
    first = None
    for _ in range(3):
        start, maps = gs.pages_extend(st, 300, slots=which, offsets=dev(np.arange(31) * 10, torch.int64))
        gs.pages_trim(st, slots=which, start=start)
        for a, b in zip(before, (st.table, st.length, st.free, st.free_count)):
            assert torch.equal(a, b)
        first = maps.clone() if first is None else first
        assert torch.equal(maps, first)


def test_no_slots_and_no_offsets():
    st, ref = gs.new_page_state(6, 20, 4, 5), du.Pages(6, 20, 4, 5)
    for _ in range(6):
        step(st, ref, [1] * 6, list(range(6)), 5, named=False)
    step(st, ref, [3, 0, 9, 2], list(range(4)), 3, named=False)
    gs.pages_trim(st, start=dev([2, 6, 4], torch.int32), keep=dev([1, 0, -9], torch.int32))
    ref.trim([0, 1, 2], [2, 6, 4], [1, 0, -9])
    check_state(st, ref)


def test_pages_run_out_in_order():
    st, ref = gs.new_page_state(2100, 1500, 4, 3), du.Pages(2100, 1500, 4, 3)
    start, rs = step(st, ref, [4] * 2100, list(range(2100)), 3)
    assert rs.count(-1) == 600
    step(st, ref, [0] * 100 + [1] * 2000, list(range(2100)), 3)
    gs.pages_trim(st)
    assert st.free_count.item() == 1500


def test_lists_that_do_not_fit_the_total():
    st = gs.new_page_state(4, 40, 4, 8)
    for offsets in ([-3, 2, 5], [0, 9, 20], [3, 1, 6], [6, 6, 6]):
        maps = torch.full((8,), -9, dtype=torch.int64, device="cuda")
        start, _ = gs.pages_extend(st, 6, offsets=dev(offsets, torch.int64), slot_map=maps[1:7])
        assert maps[0] == -9 and maps[7] == -9
        o = np.clip(offsets, 0, 6)
        counts = np.maximum(o[1:] - o[:-1], 0) if offsets != [3, 1, 6] else [0, 5]
        assert st.length[:2].tolist() == list(counts)
        gs.pages_trim(st)


def test_empty_calls_and_refusals():
    st = gs.new_page_state(4, 10, 4, 2)
    start, maps = gs.pages_extend(st, 0)
    assert start.numel() == 0 and maps.numel() == 0
    start, maps = gs.pages_extend(st, 0, offsets=torch.zeros(4, dtype=torch.int64, device="cuda"))
    assert start.tolist() == [0, 0, 0]
    i = torch.zeros(3, dtype=torch.int32, device="cuda")
    for kw in (dict(slots=i[:2]), dict(slots=i.long()), dict(slot_map=i), dict(start=i[:1]),
               dict(lengths=i.float()), dict(table=i), dict(table=torch.zeros(3, 2, device="cuda"))):
        with pytest.raises(ValueError):
            gs.pages_extend(st, 3, **kw)
    with pytest.raises(gs.GSampleError):
        gs.pages_extend(st, 5)  # more requests than slots
    with pytest.raises(ValueError):
        gs.pages_trim(st, slots=i, keep=i[:2])
    with pytest.raises(ValueError):
        gs.PageState(st.table, st.length, st.free, st.free_count, 1 << 30)
    with pytest.raises(AttributeError):
        st.table = None


def test_large_maps_pass_32_bits():
    """Slot indices past 2^31 with pages of a large pool."""
    pages, page = 300000, 16384
    st = gs.new_page_state(3, pages, page, 40)
    start, maps = gs.pages_extend(st, 3 * page, offsets=dev([0, page, 2 * page, 3 * page], torch.int64))
    st.free.copy_(torch.arange(pages, dtype=torch.int32, device="cuda"))
    st.free_count.fill_(pages)
    gs.pages_trim(st)
    st.free.copy_(torch.arange(pages, dtype=torch.int32, device="cuda"))
    st.free_count.fill_(pages)
    start, maps = gs.pages_extend(st, 3 * page, offsets=dev([0, page, 2 * page, 3 * page], torch.int64))
    want = torch.cat([torch.arange(page) + (pages - 1 - i) * page for i in range(3)])
    assert torch.equal(maps.cpu(), want) and int(maps.max()) > 1 << 32


def test_a_speculative_decode_loop():
    """Drafts verified on the GPU; the lengths, pages, histories and slot maps
    follow without the host; the same loop on the host gives the same state."""
    rng = np.random.default_rng(21)
    n, V, k, page = 9, 600, 4, 4
    slots = rng.permutation(16)[:n]
    st, ref = gs.new_page_state(16, 200, page, 20), du.Pages(16, 200, page, 20)
    hist = gs.new_logit_state(16, V, bias=False)
    sd = dev(slots, torch.int32)
    offsets = np.arange(n + 1) * (k + 1)
    od = dev(offsets, torch.int64)
    seen = np.zeros((16, V), int)
    prompt = rng.integers(1, 12, n)
    step(st, ref, prompt, slots.tolist(), 20)
    for turn in range(5):
        x = torch.from_numpy((rng.standard_normal((n * (k + 1), V)) * 3).astype(np.float32)).cuda()
        h = x.cpu().numpy()
        draft = np.where(rng.random(len(h)) < 0.7, h.argmax(1), rng.integers(0, V, len(h)))
        u, d = rng.random(len(h)).astype(np.float32), rng.random(n).astype(np.float32)
        start, maps = gs.pages_extend(st, len(h), slots=sd, offsets=od)
        tokens, count = gs.verify_drafts(x, dev(draft, torch.int64), od, 0.7,
                                         torch.from_numpy(u).cuda(), torch.from_numpy(d).cuda(),
                                         top_p=0.9)
        gs.history_append(hist, tokens, slots=sd, offsets=od)
        gs.pages_trim(st, slots=sd, start=start, keep=count)
        rs, rm, _, _ = ref.extend([k + 1] * n, slots.tolist())
        rt, rc, gaps = du.verify(h, draft, offsets, np.full(n, 0.7), u, d, p=np.full(n, 0.9))
        assert gaps.min() > 2 * du.tolerance(V)
        ref.trim(slots.tolist(), rs, rc.tolist())
        for i, s in enumerate(slots):
            for t in rt[offsets[i]:offsets[i + 1]]:
                if t >= 0:
                    seen[s, t] += 1
        assert start.tolist() == rs and maps.tolist() == sum(rm, [])
        assert tokens.tolist() == rt.tolist() and count.tolist() == rc.tolist()
        check_state(st, ref)
        assert np.array_equal(hist.history.cpu().numpy()[:, :V], seen)


def test_a_captured_step():
    st = gs.new_page_state(8, 100, 4, 12)
    sd = torch.arange(8, dtype=torch.int32, device="cuda")
    start = torch.zeros(8, dtype=torch.int32, device="cuda")
    maps = torch.zeros(24, dtype=torch.int64, device="cuda")
    keep = torch.tensor([1, 2, 3, 1, 2, 3, 1, 2], dtype=torch.int32, device="cuda")
    offsets = dev(np.arange(9) * 3, torch.int64)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gs.pages_extend(st, 24, slots=sd, offsets=offsets, slot_map=maps, start=start)
        gs.pages_trim(st, slots=sd, start=start, keep=keep)
    ref = du.Pages(8, 100, 4, 12)
    for _ in range(6):
        g.replay()
        rs, rm, _, _ = ref.extend([3] * 8, list(range(8)))
        ref.trim(list(range(8)), rs, keep.tolist())
        assert start.tolist() == rs and maps.tolist() == sum(rm, [])
        check_state(st, ref)
