"""The page plan against the list-based statement (needs a B200): whole numbers,
equal to the last one."""
import numpy as np
import pytest
import torch

import ffn_long_video_b200 as fb
from oracle import generation_ref as gen

pytestmark = pytest.mark.gpu


def _t(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


class State:
    """A pool on the device and its list-based twin."""

    def __init__(self, n, cols, page, pool, seed=0, spare_cols=0):
        r = np.random.default_rng(seed)
        self.page = page
        self.table = np.full((n, cols), -7)
        self.free, self.n_free = r.permutation(pool), pool
        wide = _t(np.full((n, cols + spare_cols), -7))
        self.d_table = wide[:, :cols]
        self.d_free, self.d_n = _t(self.free), _t([pool])
        self.lens = np.zeros(n, int)

    def step(self, new, n_rows, **kw):
        """Runs both; returns the device's slots, positions, starts, status."""
        slots, pos, starts, ws = fb.kv_plan(_t(self.lens), _t(new), self.d_table, self.d_free,
                                            self.d_n, self.page, n_rows, **kw)
        code, det = fb.read_device_status(ws)
        got = gen.kv_plan(self.lens, new, self.table, self.free, self.n_free, self.page, n_rows)
        if got is None:
            assert code == fb.EDEVICE
            assert torch.all(slots == -1) and torch.all(pos == 0) and torch.all(starts == 0)
        else:
            assert code == fb.OK, det
            self.table, self.free, self.n_free = got[:3]
            self.lens = np.array(new)
            assert slots.tolist() == got[3] and pos.tolist() == got[4]
            assert starts.tolist() == got[5]
        self.same()
        return slots, pos, starts, (code, det)

    def same(self):
        assert np.array_equal(self.d_table.cpu().numpy(), self.table)
        assert np.array_equal(self.d_free.cpu().numpy(), self.free)
        assert self.d_n.item() == self.n_free


@pytest.mark.parametrize("n,cols,page,pool", [
    (1, 5, 16, 5), (1, 300, 1, 280), (7, 12, 4, 50), (64, 9, 16, 300), (300, 6, 64, 900),
    (1023, 4, 3, 2000), (1024, 3, 16, 1700), (1025, 3, 16, 1700), (2500, 5, 2, 6000)])
def test_random_steps(n, cols, page, pool):
    """Growth by a few tokens, prompts, releases and truncations, some of them
    more than the pool holds."""
    r = np.random.default_rng(n)
    st = State(n, cols, page, pool, seed=n, spare_cols=n % 3)
    refused = 0
    for k in range(12):
        x = r.random(n)
        new = np.minimum(st.lens + r.integers(0, 4, n), cols * page)
        new = np.where(x < 0.2, 0, new)
        new = np.where((x >= 0.2) & (x < 0.5), r.integers(0, cols * page + 1, n), new)
        need = int(np.maximum(new - st.lens, 0).sum())
        *_, (code, _) = st.step(new, max(1, need + int(r.integers(0, 40))))
        refused += code != fb.OK
    assert refused < 12


def test_step_back_restores_the_pool():
    st = State(40, 20, 8, 500, seed=9)
    r = np.random.default_rng(1)
    st.step(r.integers(0, 100, 40), 5000)
    table, free, n_free, lens = st.d_table.clone(), st.d_free.clone(), st.n_free, st.lens
    st.step(np.where(np.arange(40) % 3 == 0, 0, np.minimum(lens + 30, 160)), 5000)
    st.step(lens, 5000)
    assert st.n_free == n_free and torch.equal(st.d_free[:n_free], free[:n_free])
    held = torch.arange(20)[None] < torch.from_numpy(-(-lens // 8))[:, None]
    assert torch.equal(st.d_table.cpu()[held], table.cpu()[held])


def test_pages_given_back_are_taken_in_the_same_step():
    st = State(2, 4, 16, 4)
    st.step([64, 0], 64)
    assert st.n_free == 0
    st.step([0, 64], 64)       # only the other sequence's pages are there
    st.step([16, 48], 64)      # and part of them back


@pytest.mark.parametrize("new,rows,bit", [
    ([200, 0, 0], 300, "DEV_BAD_LAYOUT"),          # longer than its table row
    ([0, -1, 0], 300, "DEV_BAD_LAYOUT"),
    ([0, 2 ** 31 - 1, 0], 300, "DEV_BAD_LAYOUT"),
    ([10, 10, 10], 29, "DEV_BAD_LAYOUT"),          # more new tokens than rows
    ([64, 64, 1], 300, "DEV_PAGES"),               # nine pages of eight
])
def test_a_plan_that_cannot_be_carried_out_changes_nothing(new, rows, bit):
    st = State(3, 4, 16, 8)
    *_, (code, det) = st.step(np.array(new), rows)
    assert code == fb.EDEVICE and det & 0xff == getattr(fb, bit)
    st.step([64, 48, 16], 200)                     # the pool is whole
    assert st.n_free == 0


def test_bad_pool_counts_and_pages_are_flagged():
    st = State(2, 4, 16, 8)
    st.step([20, 20], 40)
    for bad in (-1, 9):
        st.d_n.fill_(bad)
        *_, ws = fb.kv_plan(_t([20, 20]), _t([40, 20]), st.d_table, st.d_free, st.d_n, 16, 40)
        assert fb.read_device_status(ws) [1] & 0xff == fb.DEV_BAD_LAYOUT and st.d_n.item() == bad
    st.d_n.fill_(8)     # all pages free, and four held: giving them back cannot be
    *_, ws = fb.kv_plan(_t([20, 20]), _t([0, 0]), st.d_table, st.d_free, st.d_n, 16, 40)
    assert fb.read_device_status(ws)[1] & 0xff == fb.DEV_BAD_LAYOUT and st.d_n.item() == 8
    st.d_n.fill_(4)
    st.d_free[3] = 99   # no such page: its tokens get no slot
    slots, pos, _, ws = fb.kv_plan(_t([20, 20]), _t([40, 20]), st.d_table, st.d_free, st.d_n, 16, 20)
    assert fb.read_device_status(ws)[1] & 0xff == fb.DEV_BAD_LAYOUT
    assert slots[:12].min() >= 0 and torch.all(slots[12:] == -1)


def test_long_prompts_and_a_million_rows():
    n, page = 16, 16
    st = State(n, 4100, page, 70000)
    st.step(np.full(n, 65536), n * 65536 + 5)
    st.step(np.where(np.arange(n) % 2 == 0, 0, 65537), n)
    st.step(np.where(np.arange(n) % 2 == 0, 65536, 0), n * 65536)


def test_prompts_of_millions():
    """New tokens of one sequence past 2^21: sums in 64 bits."""
    st = State(3, 50000, 64, 60000)
    st.step([2 ** 21 + 5, 100, 0], 2 ** 21 + 200)
    st.step([2 ** 21 + 6, 0, 130], 300)
    st.step([0, 7, 2 ** 21], 2 ** 21 + 7)


def test_captured_steps_share_a_workspace():
    """Two captured steps over one pool and one workspace, replayed in turn, act
    as the same steps run one by one."""
    st = State(5, 10, 4, 50)
    st.step([3, 9, 0, 17, 8], 60)
    a, b = _t(st.lens), _t([4, 10, 12, 0, 9])
    ws = torch.empty(fb.kv_plan_workspace_bytes(5), dtype=torch.uint8, device="cuda")
    outs = [tuple(torch.empty(k, dtype=torch.int32, device="cuda") for k in (40, 40, 6))
            for _ in range(2)]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g, (x, y), o in zip(graphs, ((a, b), (b, a)), outs):
        with torch.cuda.graph(g):
            fb.kv_plan(x, y, st.d_table, st.d_free, st.d_n, 4, 40, slots=o[0], positions=o[1],
                       token_starts=o[2], workspace=ws)
    old = st.lens.copy()
    for _ in range(3):
        for g, new, o in ((graphs[0], b, outs[0]), (graphs[1], a, outs[1])):
            g.replay()
            torch.cuda.synchronize()
            got = gen.kv_plan(st.lens, new.tolist(), st.table, st.free, st.n_free, 4, 40)
            st.table, st.free, st.n_free = got[:3]
            st.lens = np.array(new.tolist())
            st.same()
            assert [x.tolist() for x in o] == [got[3], got[4], got[5]]
    assert np.array_equal(old, st.lens)


@pytest.mark.parametrize("n", [3, 1024, 1500])
def test_checks_of_plans_over_the_whole_gpu(n):
    """Many rows: refused plans change nothing, bad pages are flagged from whichever
    block meets them, the next plan clears the flag, releases fill the list again."""
    page, cols = 16, 400
    st = State(n, cols, page, 3 * cols + n)
    long = np.ones(n, int)
    long[:3] = (6000, 0, 5999)
    *_, (code, det) = st.step(long, int(long.sum()) - 1)
    assert code == fb.EDEVICE and det & 0xff == fb.DEV_BAD_LAYOUT
    *_, (code, det) = st.step(np.full(n, 6400), n * 6400 if n == 3 else 10000)
    if n > 3:
        assert code == fb.EDEVICE and det & 0xff == fb.DEV_BAD_LAYOUT
        over = np.ones(n, int)
        over[:4] = 6400                             # enough rows, too few pages
        *_, (code, det) = st.step(over, 30000)
        assert code == fb.EDEVICE and det & 0xff == fb.DEV_PAGES
    st.step(long, 16000)
    st.d_table[2, 374] = st.d_table[2, 374] + 10 ** 6     # the last page of sequence 2
    more = st.lens.copy()
    more[2] = 5999 + 1                              # its next token lies on that page
    slots, _, starts, ws = fb.kv_plan(_t(st.lens), _t(more), st.d_table, st.d_free, st.d_n, page,
                                      9000)
    assert fb.read_device_status(ws)[1] & 0xff == fb.DEV_BAD_LAYOUT
    assert starts[-1].item() == 1 and torch.all(slots == -1)
    st.d_table[2, 374] = st.d_table[2, 374] - 10 ** 6
    *_, ws = fb.kv_plan(_t(st.lens), _t(more), st.d_table, st.d_free, st.d_n, page, 9000,
                        workspace=ws)
    assert fb.read_device_status(ws)[0] == fb.OK
    *_, ws = fb.kv_plan(_t(more), _t(0 * more), st.d_table, st.d_free, st.d_n, page, 5000)
    assert fb.read_device_status(ws)[0] == fb.OK
    assert sorted(st.d_free.tolist()) == list(range(3 * cols + n)) and st.d_n.item() == 3 * cols + n


@pytest.mark.parametrize("bad", [-1, 20, 2 ** 31 - 1])
@pytest.mark.parametrize("n,rows", [(2, 1), (2, 5000), (1500, 1), (1500, 60000)])
def test_a_bad_page_given_back_is_flagged(n, rows, bad):
    """One block, the whole GPU, and more sequences than a block sums: a page that the pool
    does not have is flagged when its sequence ends or shrinks, in the plan that puts it on
    the list, not only when another sequence takes it. The plan is carried out all the same,
    which its detail tells from a refused one, and the plan back restores everything."""
    st = State(n, 6, 4, 20)
    lens = np.zeros(n, int)
    lens[0], lens[n - 1] = 22, 9                   # 6 pages and 3
    st.step(lens, max(rows, 31))
    table, free, n_free = st.d_table.clone(), st.d_free.clone(), st.n_free
    for new, at, col, give in ((0, 0, 2, 6), (11, 0, 5, 3), (0, n - 1, 0, 3)):
        to = lens.copy()
        to[at] = new
        was = table[at, col].item()
        st.d_table[at, col] = bad
        *_, ws = fb.kv_plan(_t(lens), _t(to), st.d_table, st.d_free, st.d_n, 4, rows)
        code, det = fb.read_device_status(ws)
        listed = table[at].tolist()
        listed[col] = bad
        end = -(-int(lens[at]) // 4)
        assert st.d_free[n_free:n_free + give].tolist() == listed[end - give:end][::-1]
        assert st.d_n.item() == n_free + give
        assert code == fb.EDEVICE and det & 0xff == fb.DEV_BAD_LAYOUT
        assert det >> 8 != fb.PLAN_REFUSED
        # back again: the bad page is taken, which is flagged, and the rest is as it was
        slots, pos, _, ws = fb.kv_plan(_t(to), _t(lens), st.d_table, st.d_free, st.d_n, 4,
                                       max(rows, 31))
        code, det = fb.read_device_status(ws)
        assert code == fb.EDEVICE and det & 0xff == fb.DEV_BAD_LAYOUT
        assert det >> 8 != fb.PLAN_REFUSED
        rows_back = int(lens[at]) - new
        assert torch.equal(slots[:rows_back] == -1, pos[:rows_back] // 4 == col)
        assert st.d_table[at, col].item() == bad and st.d_n.item() == n_free
        st.d_table[at, col] = was
        assert torch.equal(st.d_table, table) and torch.equal(st.d_free[:n_free], free[:n_free])
        # a plan of the same lengths is clean; a refused one says so
        *_, ws = fb.kv_plan(_t(lens), _t(lens), st.d_table, st.d_free, st.d_n, 4, rows)
        assert fb.read_device_status(ws) == (fb.OK, 0)
        *_, ws = fb.kv_plan(_t(lens), _t(lens * 0 - 1), st.d_table, st.d_free, st.d_n, 4, rows)
        assert fb.read_device_status(ws)[1] >> 8 == fb.PLAN_REFUSED
