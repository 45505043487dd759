"""Pages and slots of a batch: whole numbers, equal to the plain form's."""
import numpy as np
import pytest
import torch

import q4_weight_quantized_gb300 as q4k
from oracle import step_ref as R

GUARD = -77


def state(B, page, per, seed, over=0.1, surplus=3, spare=20, new_hi=40, odd=False):
    """Requests with pages of their own and a free list; numpy int32 arrays."""
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, (per - surplus) * page // 2 + 1, B)
    n_new = np.where(rng.random(B) < over, -1, rng.integers(0, new_hi + 1, B))
    held = np.minimum(-(-lens // page) + rng.integers(0, surplus + 1, B), per)
    n_pages = int(held.sum()) + spare + 7
    ids = rng.permutation(n_pages)
    table = np.full((B, per), GUARD)
    at = 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    free = np.full(n_pages, GUARD)
    free[:spare] = ids[at:at + spare]
    first = lens + rng.integers(0, 3, B) * 1000
    if odd:  # more pages or fewer than the length says
        held = np.maximum(held - rng.integers(0, 2, B), 0)
    return dict(table=table, lens=lens, n_new=n_new, held=held, free=free, count=spare, first=first, n_pages=n_pages, page=page, per=per)


def expect(s, T, first=True):
    return R.batch_plan(s["table"], s["per"], s["page"], s["n_pages"], s["lens"], s["n_new"], s["first"] if first else None,
                        s["held"], s["free"], s["count"], T)


def call(s, T, first=True, in_place=False, ld=None, stream=None, dev=None):
    """The call on the GPU; returns its outputs by the plain form's names."""
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
    B = len(s["lens"])
    wide = torch.full((B, ld or s["per"]), GUARD, dtype=torch.int32, device="cuda")
    wide[:, :s["per"]] = i32(s["table"])
    k = torch.zeros(s["n_pages"], 1, s["page"], 64, dtype=torch.bfloat16, device="cuda")
    cache = q4k.kv_cache(k, k, wide[:, :s["per"]])
    lens, held, count, free, new = i32(s["lens"]), i32(s["held"]), i32([s["count"]]), i32(s["free"]), i32(s["n_new"])
    pos0 = i32(s["first"]) if first else None
    fresh = lambda n: torch.full((n,), GUARD, dtype=torch.int32, device="cuda")  # noqa: E731
    after, held_out, count_out = (lens, held, count) if in_place else (fresh(B), fresh(B), fresh(1))
    starts, seq, slot, pos = fresh(B + 1), fresh(T + 4), fresh(T + 4), fresh(T + 4)
    size = q4k.q4k_batch_plan_workspace_size(cache)
    ws = torch.full((size,), 0x5A, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    q4k.q4k_batch_plan(cache, lens, new, pos0, held, held_out, free, count, count_out, T, after, starts, seq, slot, pos, ws, size,
                       stream)
    torch.cuda.synchronize()
    for a in (seq, slot, pos):
        assert (a[T:] == GUARD).all()
    assert (wide[:, s["per"]:] == GUARD).all()
    return dict(table=wide[:, :s["per"]], held=held_out, free_pages=free, count=count_out, after=after, starts=starts, seq=seq[:T],
                slot=slot[:T], pos=pos[:T])


def check(got, want, T):
    n = len(want["seq"])
    for name in ("table", "held", "free_pages", "count", "after", "starts"):
        assert np.array_equal(got[name].cpu().numpy().ravel(), np.asarray(want[name]).ravel()), name
    for name, pad in (("seq", -1), ("slot", 0), ("pos", 0)):
        a = got[name].cpu().numpy()
        assert np.array_equal(a[:n], want[name]) and (a[n:] == pad).all() and len(a) == T, name


@pytest.fixture(scope="module")
def lib():
    from q4_weight_quantized_gb300.build import build_library
    build_library()
    return q4k.load()


def test_the_plain_form_by_hand():
    # pages of 4; request 0 needs one page, 1 is over and gives two back, 2 gives one back, 3 has room
    s = dict(table=np.array([[10, 0, 0], [11, 12, 0], [13, 14, 0], [15, 0, 0]]), lens=[4, 6, 3, 1], n_new=[2, -1, 1, 0],
             held=[1, 2, 2, 1], free=np.array([20, 21, 0, 0, 0, 0]), count=2, first=[4, 6, 103, 1], n_pages=6, page=4, per=3)
    w = expect(s, 10)
    assert w["free_pages"].tolist() == [20, 21, 11, 12, 14, 0] and w["table"][0].tolist() == [10, 14, 0] and w["count"] == 4
    assert w["held"] == [2, 0, 1, 1] and w["after"] == [6, 0, 4, 1] and w["starts"].tolist() == [0, 2, 2, 3, 3]
    assert w["seq"].tolist() == [0, 0, 2] and w["slot"].tolist() == [4, 5, 3] and w["pos"].tolist() == [4, 5, 103]
    assert expect(s, 1)["seq"].tolist() == []  # request 0 has taken the sum beyond 1


CASES = [  # B, page, per, new_hi, spare, T
    (1, 16, 8, 1, 4, 1), (7, 16, 8, 1, 20, 7), (64, 16, 40, 3, 100, 300), (33, 1, 200, 60, 4000, 2000), (200, 24, 30, 90, 1000, 9000),
    (1024, 16, 20, 9, 1500, 6000), (1025, 64, 9, 50, 900, 40000), (3000, 16, 12, 30, 4000, 100000), (5000, 128, 5, 1, 300, 5000)]


@pytest.mark.gpu
@pytest.mark.parametrize("B,page,per,new_hi,spare,T", CASES)
@pytest.mark.parametrize("short", [False, True])
def test_plan(lib, B, page, per, new_hi, spare, T, short):
    s = state(B, page, per, B + page, spare=spare // 8 if short else spare, new_hi=new_hi)
    T = max(1, int(np.maximum(s["n_new"], 0).sum() * 0.7)) if short else T
    check(call(s, T), expect(s, T), T)
    check(call(s, T, first=False, in_place=True, ld=per + 3), expect(s, T, first=False), T)
    q4k.q4k_check_device()


@pytest.mark.gpu
def test_plan_requests_without_tokens_and_none_at_all(lib):
    s = state(50, 16, 10, 3, over=0.0, new_hi=0)
    check(call(s, 5), expect(s, 5), 5)
    s = state(50, 16, 10, 4, over=1.0)
    check(call(s, 5), expect(s, 5), 5)
    s = state(30, 8, 10, 5, spare=0, surplus=0)
    check(call(s, 900), expect(s, 900), 900)
    s = state(40, 8, 20, 6, odd=True)
    check(call(s, 2000), expect(s, 2000), 2000)
    q4k.q4k_check_device()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3000, 20000])
def test_plan_out_of_range(lib, T):
    """Lengths, held pages, token counts and a list's length out of range, and a page id that changes hands."""
    def bad(change, **a):
        s = state(60, 16, 12, 9, **a)
        change(s)
        check(call(s, T), expect(s, T), T)
        with pytest.raises(q4k.Q4KError) as e:
            q4k.q4k_check_device()
        assert e.value.status == q4k.Q4K_ERR_INDEX
    def put(name, i, v):
        def f(s):
            s[name][i] = v
        return f
    bad(put("lens", 3, -4))
    bad(put("lens", 3, 12 * 16 + 1))
    bad(put("held", 5, -1))
    bad(put("n_new", 7, 12 * 16 + 1))
    bad(put("n_new", 7, 2 ** 31 - 1))
    bad(lambda s: s.update(count=-3))
    bad(put("free", 19, 10 ** 6), over=0.0, surplus=0)  # (nothing comes back: the list's end is handed out)
    def over_and_bad(s):
        s["n_new"][0], s["held"][0] = -1, max(1, s["held"][0])
        s["table"][0, 0] = -5
    bad(over_and_bad)
    def full(s):  # a list that says it is full, and pages coming back
        s["count"], s["n_new"][1], s["held"][1], s["lens"][1] = s["n_pages"], -1, 2, 20
        s["table"][1, :2] = [1, 2]
        s["free"][:] = np.arange(s["n_pages"])
    bad(full)


@pytest.mark.gpu
def test_plan_most_requests(lib):
    s = state(65535, 16, 3, 1, surplus=1, new_hi=4, spare=50000)
    check(call(s, 200000), expect(s, 200000), 200000)
    q4k.q4k_check_device()


@pytest.mark.gpu
def test_plan_on_another_stream_and_in_a_graph(lib):
    s = state(70, 16, 30, 2, spare=400)
    side = torch.cuda.Stream()
    check(call(s, 3000, stream=side), expect(s, 3000), 3000)
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
    table, lens, held, count, free, new = (i32(s[n]) for n in ("table", "lens", "held", "count", "free", "n_new"))
    count = count.view(1)
    k = torch.zeros(s["n_pages"], 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    cache = q4k.kv_cache(k, k, table)
    starts, seq, slot, pos = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (71, 3000, 3000, 3000))
    ws = torch.empty(q4k.q4k_batch_plan_workspace_size(cache), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        q4k.q4k_batch_plan(cache, lens, new, None, held, held, free, count, count, 3000, lens, starts, seq, slot, pos, ws, ws.numel())
    for step in range(4):  # each replay goes on from what the last one left
        want = R.batch_plan(table.cpu().numpy(), 30, 16, s["n_pages"], lens.tolist(), new.tolist(), None, held.tolist(),
                            free.cpu().numpy(), int(count), 3000)
        graph.replay()
        torch.cuda.synchronize()
        check(dict(table=table, held=held, free_pages=free, count=count, after=lens, starts=starts, seq=seq, slot=slot, pos=pos),
              want, 3000)
        new.copy_(torch.where(new < 0, torch.ones_like(new), torch.full_like(new, 17 if step else -1)))
    q4k.q4k_check_device()
