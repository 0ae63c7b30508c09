"""Eviction against the rule on the host: every array bit for bit, ties, protected rows, NaN, pages, lengths of the batch."""
import numpy as np
import pytest
import torch

import attention_quantized_kv_split_gb300 as qda

import forget_ref as R

pytestmark = pytest.mark.gpu


class Pool:
    def __init__(self, kv, Hkv=2, D=64, bits=4, GS=32, page=16, seed=0, spare=3, extra_cols=1, order="scattered", ties=False):
        rng = np.random.default_rng(seed)
        need = [-(-n // page) for n in kv]
        pool = sum(need) + spare
        ids = rng.permutation(pool).astype(np.int32)
        self.kv, self.page, self.Hkv, self.GS, self.bits = np.array(kv, dtype=np.int32), page, Hkv, GS, bits
        self.table = np.full((len(kv), max(need + [1]) + extra_cols), -1, dtype=np.int32)
        self.shift = (rng.integers(0, 50, len(kv)) if order == "scattered" else np.zeros(len(kv))).astype(np.int32)
        rows = (pool, Hkv, page)
        self.mass = rng.random(rows).astype(np.float32)
        if ties:
            self.mass = np.floor(self.mass * 4) / 4
        self.token = rng.integers(0, 1 << 30, rows).astype(np.int32)
        at = 0
        for b, m in enumerate(need):
            self.table[b, :m] = ids[at: at + m]
            at += m
            n = kv[b]
            for h in range(Hkv):
                tok = np.arange(n) if order == "fresh" else rng.permutation(n) + self.shift[b]
                i = np.arange(n)
                self.token[self.table[b][i // page], h, i % page] = tok
        W, NG = D * bits // 32, D // GS
        words = lambda: rng.integers(-(1 << 31), 1 << 31, (*rows, W), dtype=np.int64).astype(np.int32)  # noqa: E731
        half = lambda: rng.integers(-(1 << 15), 1 << 15, (*rows, NG), dtype=np.int64).astype(np.int16)  # noqa: E731
        self.arrays = [words(), half(), half(), words(), half(), half()]

    def run(self, budget, limit=None, sinks=0, recent=0, shift=True, max_freed=None, stream=None, device="cuda"):
        put = lambda a: torch.from_numpy(np.array(a)).to(device)  # noqa: E731
        arrays = [put(a) for a in self.arrays]
        arrays = [a if a.dtype == torch.int32 else a.view(torch.bfloat16) for a in arrays]
        self.dev = dict(arrays=arrays, mass=put(self.mass), token=put(self.token), kv=put(self.kv), table=put(self.table),
                        new=put(self.kv * 0 - 7), shift=put(self.shift) if shift else None,
                        freed=torch.full((self.table.size if max_freed is None else max_freed,), -7, dtype=torch.int32, device=device),
                        n_freed=torch.full((1,), -7, dtype=torch.int32, device=device))
        self.call(budget, limit, sinks, recent, stream)
        torch.cuda.synchronize()
        return self.got()

    def call(self, budget, limit, sinks, recent, stream=None):
        d = self.dev
        qda.qdecode_paged_evict(*d["arrays"], d["mass"], d["token"], d["kv"], d["new"], d["table"], d["freed"], d["n_freed"], self.GS,
                                self.bits, budget, limit, sinks, recent, d["shift"], stream)

    def got(self):
        d = self.dev
        n = lambda t: None if t is None else t.cpu().numpy()  # noqa: E731
        arrays = [n(a if a.dtype == torch.int32 else a.view(torch.int16)) for a in d["arrays"]]
        return arrays, n(d["mass"]), n(d["token"]), n(d["new"]), n(d["table"]), n(d["freed"]), int(d["n_freed"]), n(d["shift"])

    def check(self, budget, limit=None, sinks=0, recent=0, shift=True, max_freed=None, **kw):
        got = self.run(budget, limit, sinks, recent, shift, max_freed, **kw)
        freed = np.full(self.table.size if max_freed is None else max_freed, -7)
        want = R.evict(self.arrays, self.mass, self.token, self.kv, self.table, freed, self.page, budget, limit, sinks, recent,
                       self.shift if shift else None)
        for a, b in zip(got[0], want[0]):
            np.testing.assert_array_equal(a, b)
        for i, name in enumerate(("mass", "token", "new_len", "table", "freed", "n_freed", "shift"), 1):
            if want[i] is not None:
                np.testing.assert_array_equal(got[i], want[i], err_msg=name)


@pytest.fixture(autouse=True)
def clean_status():
    qda.qdecode_attn_device_status()
    yield
    assert qda.qdecode_attn_device_status() == 0


@pytest.mark.parametrize("kv,budget,limit", [([1], 1, None), ([2], 1, None), ([17], 16, None), ([65, 64, 1, 0, 200], 64, None),
                                             ([300, 299, 120], 100, 299), ([1000], 37, None), ([5000, 3000, 40], 2100, None)])
@pytest.mark.parametrize("ties", [False, True])
def test_sizes(kv, budget, limit, ties):
    Pool(kv, seed=sum(kv), ties=ties).check(budget, limit)


@pytest.mark.parametrize("D,bits,GS,page", [(64, 4, 32, 16), (64, 4, 64, 32), (128, 4, 128, 64), (128, 8, 32, 256), (256, 8, 64, 16),
                                            (512, 8, 32, 32), (512, 4, 128, 16), (256, 4, 32, 128)])
def test_row_layouts(D, bits, GS, page):
    Pool([333, 100, 150], Hkv=3, D=D, bits=bits, GS=GS, page=page, seed=D).check(99, 110, 2, 5)


@pytest.mark.parametrize("order", ["scattered", "fresh"])
@pytest.mark.parametrize("sinks,recent", [(0, 0), (4, 0), (0, 30), (4, 60), (20, 44), (0, 64)])
def test_protected_rows(order, sinks, recent):
    """Up to the whole budget of protected rows, wherever they stand."""
    Pool([200, 130, 64], seed=sinks + recent, order=order).check(64, None, sinks, recent)


@pytest.mark.parametrize("shift", [True, False])
def test_tokens_without_a_shift(shift):
    Pool([150, 90], order="fresh", seed=9).check(70, None, 3, 10, shift)


def test_masses_that_are_no_numbers_or_all_alike():
    p = Pool([200, 200, 200, 200], seed=3)
    for b, v in ((0, np.nan), (1, 0.0), (2, np.inf)):
        p.mass[p.table[b][np.arange(200) // 16], :, np.arange(200) % 16] = v
    pg, row = p.table[3][np.arange(200) // 16], np.arange(200) % 16
    p.mass[pg, :, row] = np.random.default_rng(0).choice([np.nan, -np.inf, -1.0, -0.5, 1e-45, 0.5, np.inf], (200, 2))
    p.check(90, None, 1, 3)


def test_many_heads_of_many_sequences():
    rng = np.random.default_rng(5)
    Pool([int(n) for n in rng.integers(0, 120, 130)], Hkv=4, seed=5, ties=True).check(60, 70, 1, 8)


@pytest.mark.parametrize("n,budget", [(70000, 3000), (40000, 39990), (140000, 70000)])
def test_long_rows_over_a_cluster(n, budget):
    """Pieces of a head beyond what a CTA holds in shared memory, compared with a stable sort."""
    p = Pool([n], Hkv=1, page=256, seed=n, order="fresh", ties=budget == 70000)
    got = p.run(budget, None, 4, 100)
    i = np.arange(n)
    pg, row = p.table[0][i // 256], i % 256
    m = p.mass[pg, 0, row].astype(np.float64)
    m[:4] = m[n - 100:] = np.inf
    kept = np.argsort(-m, kind="stable")[:budget]
    stay = np.zeros(n, bool)
    stay[kept] = True
    holes, comes = np.flatnonzero(~stay[:budget]), budget + np.flatnonzero(stay[budget:])
    src = i.copy()[:budget]
    src[holes] = comes
    np.testing.assert_array_equal(got[2][pg[:budget], 0, row[:budget]], src)
    for a, b in zip((*got[0], got[1]), (*p.arrays, p.mass)):
        np.testing.assert_array_equal(a[pg[:budget], 0, row[:budget]], b[pg[src], 0, row[src]])
    assert got[3][0] == budget and got[6] == -(-n // 256) - -(-budget // 256)


def test_nothing_else_is_touched():
    """Rows of sequences that are not cut, pages of nobody, and table entries that stay."""
    p = Pool([100, 30, 64], seed=12, spare=5)
    got = p.run(40, 64)
    used = np.zeros(p.mass.shape[0], bool)
    used[p.table[0][:7]] = True
    for a, b in zip((*got[0], got[1], got[2]), (*p.arrays, p.mass, p.token)):
        np.testing.assert_array_equal(a[~used], b[~used])
    np.testing.assert_array_equal(got[4][1:], p.table[1:])
    np.testing.assert_array_equal(got[3], [40, 30, 64])


def test_pages_that_find_no_place():
    Pool([100, 100], seed=2).check(20, max_freed=3)
    assert qda.qdecode_attn_device_status() == 8


def test_bad_lengths_leave_their_sequence():
    p = Pool([100, 100, 100], seed=4)
    cols = p.table.shape[1]
    p.kv[0], p.kv[2] = -3, cols * 16 + 1
    got = p.run(50)
    assert qda.qdecode_attn_device_status() == 8
    np.testing.assert_array_equal(got[3], [-3, 50, cols * 16 + 1])
    np.testing.assert_array_equal(got[4][[0, 2]], p.table[[0, 2]])
    np.testing.assert_array_equal(got[7] - p.shift, [0, 50, 0])


def test_absent_pages_are_neither_read_nor_written():
    p = Pool([100], seed=6, spare=4)
    p.table[0, 1], p.table[0, 5] = -1, p.mass.shape[0]
    got = p.run(50)
    assert qda.qdecode_attn_device_status() == 8
    used = np.zeros(p.mass.shape[0], bool)
    used[p.table[0][[0, 2, 3, 4, 6]]] = True
    for a, b in zip((*got[0], got[1], got[2]), (*p.arrays, p.mass, p.token)):
        np.testing.assert_array_equal(a[~used], b[~used])
    assert got[3][0] == 50


@pytest.mark.parametrize("kv,Hkv,budget", [([300, 700], 2, 64), ([9000], 1, 4000)])
def test_own_workspace_is_enough_and_nothing_else_is_touched(kv, Hkv, budget):
    p = Pool(kv, Hkv=Hkv, seed=31)
    need = qda.qdecode_paged_evict_workspace_bytes(len(kv), Hkv, 16, p.table.shape[1], budget)
    buf = torch.full((need + 8192,), 0x5A, dtype=torch.uint8, device="cuda")
    try:
        qda.qdecode_attn_set_workspace(buf[4096: 4096 + need])
        p.check(budget, None, 1, 3)
        qda.qdecode_attn_set_workspace(buf[4096: 4096 + need - 16])
        with pytest.raises(qda.QdaError, match="-5"):
            p.call(budget, None, 1, 3)
    finally:
        qda.qdecode_attn_set_workspace(None)
    assert bool((buf[:4096] == 0x5A).all()) and bool((buf[4096 + need:] == 0x5A).all())


def test_masses_whose_leading_bits_agree():
    """Rows that differ in the last bits of their masses alone, and many that do not differ at all: more of them than are
    compared one by one, so that every pass over the bits, and then the rows' order, decides."""
    p = Pool([1500, 1500, 1500], Hkv=1, seed=40, page=32)
    rng = np.random.default_rng(8)
    i = np.arange(1500)
    for b, bits in enumerate((rng.integers(0, 4, 1500), rng.integers(0, 1500, 1500), np.where(rng.random(1500) < 0.8, 7, rng.integers(0, 14, 1500)))):
        p.mass[p.table[b][i // 32], 0, i % 32] = (np.float32(1.0).view(np.int32) + bits.astype(np.int32)).view(np.float32)
    p.check(700, None, 0, 0)


def test_other_calls_between_do_not_matter():
    """The lists in the workspace are a call's own: evictions of other pools and attention between two alike."""
    a, b = Pool([400, 300], seed=50), Pool([5000], Hkv=4, seed=51, page=64)
    first = a.run(100, None, 2, 9)
    b.check(2500)
    again = a.run(100, None, 2, 9)
    for x, y in zip((*first[0], *first[1:6]), (*again[0], *again[1:6])):
        np.testing.assert_array_equal(x, y)


def test_graph_stream_and_growing_batches():
    """A captured call replayed on other weights, with a larger call (and workspace) between."""
    p = Pool([300, 120], seed=21)
    p.check(64, None, 2, 8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    p.check(64, None, 2, 8, stream=s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.call(64, None, 2, 8)
    Pool([3000] * 6, Hkv=4, seed=1).check(1500)
    p.mass = np.random.default_rng(3).random(p.mass.shape).astype(np.float32)
    for k, v in (("mass", p.mass), ("token", p.token), ("kv", p.kv), ("table", p.table), ("shift", p.shift)):
        p.dev[k].copy_(torch.from_numpy(np.array(v)))
    for d, a in zip(p.dev["arrays"], p.arrays):
        d.copy_(torch.from_numpy(a) if a.dtype == np.int32 else torch.from_numpy(a).view(torch.bfloat16))
    p.dev["freed"].fill_(-7)
    g.replay()
    torch.cuda.synchronize()
    got = p.got()
    want = R.evict(p.arrays, p.mass, p.token, p.kv, p.table, np.full(p.table.size, -7), 16, 64, None, 2, 8, p.shift)
    for a, b in zip(got[0], want[0]):
        np.testing.assert_array_equal(a, b)
    for a, b in zip(got[1:], want[1:]):
        np.testing.assert_array_equal(a, b)


def test_zeros_of_either_sign_are_alike():
    """-0.0 and 0.0 are equal masses: of them the lowest rows stay."""
    p = Pool([200, 3000], Hkv=2, seed=60, page=32)
    p.mass[:] = np.random.default_rng(4).choice(np.array([-0.0, 0.0], dtype=np.float32), p.mass.shape)
    p.mass[p.table[1, :9]] = np.float32(-1e-45)
    p.check(70, None, 1, 3)


@pytest.mark.parametrize("recent", [0, 1, 7])
def test_newest_position_of_all(recent):
    """Tokens up to position 2^31 - 1: those that are protected are the newest, none where none is asked for."""
    p = Pool([200], seed=61)
    p.shift[:] = (1 << 31) - 200   # (the newest token's position is 2^31 - 1)
    i = np.arange(200)
    for h in range(2):
        p.token[p.table[0][i // 16], h, i % 16] = np.random.default_rng(h).permutation(200) + np.int64(p.shift[0])
    got = p.run(64, None, 0, recent)
    want = R.evict(p.arrays, p.mass, p.token, [200], p.table, np.full(p.table.size, -7), 16, 64, None, 0, recent, p.shift.astype(np.int64))
    for a, b in zip((*got[0], *got[1:]), (*want[0], *want[1:])):
        np.testing.assert_array_equal(a, b)


@pytest.mark.parametrize("kv,gone", [([100, 100], [(0, 5), (1, 4), (1, 1)]), ([100, 6000, 40, 9000], [(b, c) for b in (1, 3) for c in range(5, 375, 3)]),
                                     ([100], [(0, 4), (0, 5), (0, 6)])])
@pytest.mark.parametrize("max_freed", [None, 2])
def test_absent_pages_are_not_given_back(kv, gone, max_freed):
    """Entries outside the pool leave the table, but they are no pages: neither in freed nor counted."""
    p = Pool(kv, seed=62, spare=4)
    for j, (b, c) in enumerate(gone):
        p.table[b, c] = (-1, p.mass.shape[0], -(1 << 31))[j % 3]
    got = p.run(50, max_freed=max_freed)
    assert qda.qdecode_attn_device_status() == 8
    behind = [p.table[b, 4: -(-n // 16)] for b, n in enumerate(kv) if n > 50]
    pages = np.concatenate([x[(x >= 0) & (x < p.mass.shape[0])] for x in behind])
    assert got[6] == len(pages)
    room = p.table.size if max_freed is None else max_freed
    np.testing.assert_array_equal(got[5], np.concatenate([pages, np.full(room, -7)])[:room])
    for b, n in enumerate(kv):
        if n > 50:
            assert (got[4][b, 4:] == -1).all()
