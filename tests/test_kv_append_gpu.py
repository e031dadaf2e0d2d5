"""GPU parity of the paged cache's slots and append: values bit for bit, keys and queries within derived bounds."""
import pytest
import torch

import block_ops_ref as ref

pytestmark = pytest.mark.gpu


def _step(lens, new, page, seed, padding=0, spare=2, first=0):
    """CPU: (page_table, cache_lens, seq_starts, T, num_pages) of sequences with these lengths."""
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    most = max([1] + [-(-(a + n) // page) for a, n in zip(lens, new)]) + 1
    pages = B * most + spare
    table = torch.randperm(pages, generator=g)[: B * most].view(B, most).to(torch.int32)
    starts = torch.tensor([first] + [first + sum(new[: i + 1]) for i in range(B)], dtype=torch.int32)
    return table, torch.tensor(lens, dtype=torch.int32), starts, int(starts[-1]) + padding, pages


def _slots(ce, table, lens, starts, T, page, pages, **how):
    return ce.foak_kv_slots(table.cuda(), lens.cuda(), starts.cuda(), T, page_size=page, num_pages=pages, **how)


@pytest.mark.parametrize("page", [1, 16, 48, 7])
@pytest.mark.parametrize("lens,new,padding,first", [
    ([0], [1], 0, 0), ([5], [1], 3, 0), ([0, 15, 16, 17], [1, 1, 1, 1], 0, 2), ([31, 0, 200], [40, 1, 77], 5, 0),
    ([3, 9, 9, 0], [0, 5, 0, 0], 2, 0), ([100] * 300, [1] * 300, 7, 0), ([0], [0], 4, 0)])
def test_slots(cuda_lib, lens, new, padding, first, page):
    table, cl, starts, T, pages = _step(lens, new, page, seed=page, padding=padding, first=first)
    out = _slots(cuda_lib, table, cl, starts, T, page, pages)
    at, pos, bad = ref.slots(table, cl, starts, T, page, pages)
    assert not bad and out["slots"].tolist() == at and out["positions"].tolist() == pos and int(out["err"]) == 0


def test_slots_of_bad_tables(cuda_lib):
    """Pages that are missing, negative or too large; negative lengths; starts that are not ascending."""
    ce, page = cuda_lib, 4
    table = torch.tensor([[0, 1], [-1, 2], [9, 3], [4, 5]], dtype=torch.int32)
    lens, starts = torch.tensor([5, 0, 0, -3], dtype=torch.int32), torch.tensor([0, 5, 8, 10, 12], dtype=torch.int32)
    out = _slots(ce, table, lens, starts, 12, page, 6)
    at, pos, bad = ref.slots(table, lens, starts, 12, page, 6)
    assert bad and int(out["err"]) == ce.FOAK_ERRBIT_PAGE_RANGE
    assert out["slots"].tolist() == at and out["positions"].tolist() == pos
    err = torch.tensor([2], dtype=torch.int32, device="cuda")
    again = _slots(ce, table, lens, starts, 12, page, 6, err=err)
    assert again["err"] is err and int(err) == 2 | ce.FOAK_ERRBIT_PAGE_RANGE  # OR-ed in
    messy = _slots(ce, table, torch.tensor([0, 0, 0, 0], dtype=torch.int32), torch.tensor([3, 9, 2, 11, 4], dtype=torch.int32), 12, page, 6)
    assert all(-1 <= s < 24 for s in messy["slots"].tolist())


@pytest.mark.parametrize("B", [4095, 4096, 5000])
def test_slots_of_many_sequences(cuda_lib, B):
    """As many starts as one block keeps at hand, and more."""
    g = torch.Generator().manual_seed(B)
    lens, new = torch.randint(0, 40, (B,), generator=g).tolist(), torch.randint(0, 3, (B,), generator=g).tolist()
    table, cl, starts, T, pages = _step(lens, new, 16, seed=B, padding=300)
    out = _slots(cuda_lib, table, cl, starts, T, 16, pages)
    at, pos, bad = ref.slots(table, cl, starts, T, 16, pages)
    assert not bad and out["slots"].tolist() == at and out["positions"].tolist() == pos and int(out["err"]) == 0


def test_slots_without_sequences_or_tokens(cuda_lib):
    empty = torch.zeros(0, 3, dtype=torch.int32), torch.zeros(0, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    out = _slots(cuda_lib, *empty, 5, 16, 4)
    assert out["slots"].tolist() == [-1] * 5 and out["positions"].tolist() == [0] * 5 and int(out["err"]) == 0
    assert _slots(cuda_lib, *empty, 0, 16, 4)["slots"].numel() == 0


def _check_append(ce, lens, new, page, Hq, Hk, d, dv, r, dtype, heads_first, interleaved, padding=3, seed=1, with_q=True, far=0):
    g = torch.Generator().manual_seed(seed)
    dt = ref.DT[dtype]
    table, cl, starts, T, pages = _step(lens, new, page, seed, padding)
    at = _slots(ce, table, cl, starts, T, page, pages)
    qkv = torch.randn(T, (Hq + Hk) * d + Hk * dv, generator=g).to(dt)
    q, k, v = qkv[:, : Hq * d].unflatten(1, (Hq, d)), qkv[:, Hq * d : (Hq + Hk) * d].unflatten(1, (Hk, d)), qkv[:, (Hq + Hk) * d :].unflatten(1, (Hk, dv))
    shape = lambda n: (pages, Hk, page, n) if heads_first else (pages, page, Hk, n)  # noqa: E731
    kc, vc = torch.randn(*shape(d), generator=g).to(dt), torch.randn(*shape(dv), generator=g).to(dt)
    plan = ce.foak_rotary_plan(r, interleaved=interleaved) if r else None
    pos = at["positions"] + far if r else None
    dev = qkv.cuda()
    qd, kd, vd = dev[:, : Hq * d].unflatten(1, (Hq, d)), dev[:, Hq * d : (Hq + Hk) * d].unflatten(1, (Hk, d)), dev[:, (Hq + Hk) * d :].unflatten(1, (Hk, dv))
    kcd, vcd = kc.cuda(), vc.cuda()
    q_out = torch.full((T, Hq, d), 5.0, dtype=dt, device="cuda") if with_q and r else None
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = ce.foak_kv_append(kd, vd, kcd, vcd, at["slots"], heads_first=heads_first, plan=plan, positions=pos, q=qd if q_out is not None else None, q_out=q_out, err=err)
    assert got is q_out and int(err) == 0 and torch.equal(dev.cpu(), qkv)
    slots, positions = at["slots"].tolist(), (at["positions"] + far).tolist()
    rows = [t for t in range(T) if slots[t] >= 0]
    where = torch.tensor([slots[t] for t in rows], dtype=torch.int64)
    turns = [t % 2 ** 64 for t in plan.turns.tolist()] if r else []
    sel = [positions[t] for t in rows]

    def places(cache):  # [slots, Hk, n]
        c = cache.cpu()
        return (c.transpose(1, 2) if heads_first else c).reshape(pages * page, Hk, c.shape[-1])

    new_k, new_v = places(kcd), places(vcd)
    if rows:
        if r:
            ref.assert_close(new_k[where], ref.rotate(k[rows], sel, turns, r, interleaved), "k_cache")
        else:
            assert torch.equal(new_k[where], k[rows])
        assert torch.equal(new_v[where], v[rows])
    other = torch.ones(pages * page, dtype=torch.bool)
    other[where] = False
    assert torch.equal(new_k[other], places(kc)[other]) and torch.equal(new_v[other], places(vc)[other])
    if q_out is not None:
        if rows:
            ref.assert_close(q_out[rows], ref.rotate(q[rows], sel, turns, r, interleaved), "q")
        pad = [t for t in range(T) if slots[t] < 0]
        assert bool((q_out[pad] == 5.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("Hq,Hk,d,dv,r,interleaved", [
    (4, 1, 128, 128, 128, False), (8, 2, 128, 64, 64, True), (6, 3, 80, 80, 20, False), (5, 5, 64, 128, 64, True),
    (3, 1, 18, 10, 12, False), (2, 2, 7, 5, 6, True), (40, 8, 96, 96, 48, True), (4, 2, 256, 256, 256, False)])
def test_append(cuda_lib, Hq, Hk, d, dv, r, interleaved, heads_first, dtype):
    for lens, new, page in (([9], [1], 16), ([0, 33, 7], [50, 1, 12], 16), ([3, 0, 0, 12], [1, 9, 0, 1], 5)):
        _check_append(cuda_lib, lens, new, page, Hq, Hk, d, dv, r, dtype, heads_first, interleaved)


def test_append_forms(cuda_lib):
    ce = cuda_lib
    _check_append(ce, [4, 80], [3, 20], 16, 4, 2, 64, 64, 0, "bf16", False, False)  # no rotation
    _check_append(ce, [4, 80], [3, 20], 16, 4, 2, 64, 64, 64, "bf16", False, False, with_q=False)
    _check_append(ce, [4, 80], [3, 20], 1, 4, 2, 64, 64, 32, "f32", True, False)  # a token a page
    _check_append(ce, [0] * 200, [1] * 200, 32, 8, 2, 128, 128, 128, "bf16", False, False, padding=56)
    _check_append(ce, [2], [1], 16, 4, 2, 64, 64, 64, "f32", False, False, far=10 ** 9)  # positions of their own
    _check_append(ce, [0], [0], 16, 4, 2, 64, 64, 64, "f32", False, False, padding=4)  # padding alone


def test_many_tokens(cuda_lib):
    _check_append(cuda_lib, [100, 0, 1000], [1500, 1, 900], 64, 12, 4, 128, 128, 128, "bf16", False, False)


def test_slots_past_the_cache_are_left_out(cuda_lib):
    ce = cuda_lib
    plan = ce.foak_rotary_plan(64)
    k = torch.randn(5, 2, 64, device="cuda")
    kc, vc = torch.zeros(3, 4, 2, 64, device="cuda"), torch.zeros(3, 4, 2, 64, device="cuda")
    slots = torch.tensor([0, 12, -1, 2 ** 40, 11], device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pos = torch.zeros(5, dtype=torch.int64, device="cuda")
    ce.foak_kv_append(k, k, kc, vc, slots, plan=plan, positions=pos, err=err)
    assert int(err) == ce.FOAK_ERRBIT_PAGE_RANGE
    flat = vc.view(12, 2, 64)
    assert torch.equal(flat[0], k[0]) and torch.equal(flat[11], k[4]) and not flat[1:11].any()
    ce.foak_kv_append(k, k, kc, vc, slots, plan=plan, positions=pos)  # nobody asks


def test_queries_in_place_and_caches_as_views(cuda_lib):
    """One tensor of keys and values, pages first; queries rotated where they are."""
    ce = cuda_lib
    plan = ce.foak_rotary_plan(32)
    both = torch.zeros(6, 2, 8, 2, 64, device="cuda")
    q, k, v = (torch.randn(3, h, 64, device="cuda") for h in (4, 2, 2))
    slots, pos = torch.tensor([5, 40, 47], device="cuda"), torch.tensor([9, 1, 4], device="cuda")
    want = ce.foak_rotary_apply(plan, pos, q, k)
    out = ce.foak_kv_append(k, v, both[:, 0], both[:, 1], slots, plan=plan, positions=pos, q=q, q_out=q)
    assert out is q and torch.equal(q, want[0])
    flat = both.transpose(0, 1).reshape(2, 48, 2, 64)
    assert torch.equal(flat[0][slots], want[1]) and torch.equal(flat[1][slots], v)
    assert int((flat != 0).any(-1).any(-1).sum()) == 6


def test_offsets_past_32_bits(cuda_lib):
    """A cache of more than 2^32 elements: its last pages."""
    ce = cuda_lib
    page, Hk, d = 64, 8, 128
    pages = 2 ** 32 // (page * Hk * d) + 3
    kc = torch.empty(pages, page, Hk, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    kc[-1], vc[-1], kc[0], vc[0] = 0, 0, 0, 0
    k = torch.randn(2, Hk, d, device="cuda").bfloat16()
    slots = torch.tensor([pages * page - 1, pages * page - 7], device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ce.foak_kv_append(k, k, kc, vc, slots, err=err)
    for c in (kc, vc):
        assert torch.equal(c[-1, [63, 57]], k) and not c[-1, :57].any() and not c[0].any()
    assert int(err) == 0


def test_refusals_of_the_binding(cuda_lib):
    ce = cuda_lib
    plan = ce.foak_rotary_plan(64)
    k = torch.zeros(3, 2, 64, device="cuda")
    c, c2 = torch.zeros(4, 16, 2, 64, device="cuda"), torch.zeros(4, 16, 2, 64, device="cuda")
    s = torch.zeros(3, dtype=torch.int64, device="cuda")
    i32 = lambda *shape: torch.zeros(*shape, dtype=torch.int32, device="cuda")  # noqa: E731
    bad = [
        lambda: ce.foak_kv_append(k, k[:, :1], c, c2, s),
        lambda: ce.foak_kv_append(k, k[:2], c, c2, s),
        lambda: ce.foak_kv_append(k, k, c, c2[:3], s),
        lambda: ce.foak_kv_append(k, k, c.bfloat16(), c2, s),
        lambda: ce.foak_kv_append(k, k, c, c2, s[:2]),
        lambda: ce.foak_kv_append(k, k, c, c2, s.int()),
        lambda: ce.foak_kv_append(k, k, c, c2, s, heads_first=True),
        lambda: ce.foak_kv_append(k, k, c, c2, s, plan=plan),
        lambda: ce.foak_kv_append(k, k, c, c2, s, q=k),
        lambda: ce.foak_kv_append(k, k, c, c2, s, q_out=k),
        lambda: ce.foak_kv_append(k, k, c, c2, s, err=torch.zeros(1, dtype=torch.int32)),
        lambda: ce.foak_kv_append(k, k, c[0], c2, s),
        lambda: ce.foak_kv_slots(i32(2, 4), i32(2), i32(2), 3, page_size=16, num_pages=4),
        lambda: ce.foak_kv_slots(i32(2, 4), i32(3), i32(3), 3, page_size=16, num_pages=4),
        lambda: ce.foak_kv_slots(i32(2, 4).long(), i32(2), i32(3), 3, page_size=16, num_pages=4),
        lambda: ce.foak_kv_slots(i32(2, 4).cpu(), i32(2), i32(3), 3, page_size=16, num_pages=4),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was taken")
    for call in (lambda: ce.foak_kv_append(k, k, c, c, s),
                 lambda: ce.foak_kv_append(k, k, c[:1].expand(4, 16, 2, 64), c2, s),
                 lambda: ce.foak_kv_slots(i32(2, 4), i32(2), i32(3), 3, page_size=0, num_pages=4)):
        with pytest.raises(ce.FoakError):
            call()
