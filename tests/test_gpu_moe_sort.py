"""The dispatch's sort past the slots whose block counts every block may sum for itself (524288): against a stable sort,
rows and split sizes exact, and its time in proportion to the slots."""

import pytest


def test_scratch_has_a_row_of_totals_past_128_blocks():
    """(On the CPU.)  Counts per block of 4096 slots and expert, and the experts' totals where a launch sums them."""
    from moe_grouped_scaled_amd import _native as N
    need = N.LIB.mgs_moe_dispatch_workspace_bytes
    assert need(524288, 1, 37) == 4 * 128 * 37
    assert need(524289, 1, 37) == 4 * (129 + 1) * 37
    assert need((1 << 28) - 1, 8, 256) == 4 * (524288 + 1) * 256


def _picks(t, k, e, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    # unequal shares, some slots without an expert and some entries outside the experts
    x = torch.rand((t, k), generator=g, device="cuda")
    idx = (x * x * (e + 2)).to(torch.int32) - 1
    return torch.where(idx >= e, 2 ** 31 - 1, idx).to(torch.int32)


@pytest.mark.gpu
@pytest.mark.parametrize("t,k,e", [(131072, 4, 256), (131073, 4, 256), (524289, 1, 1), (174763, 3, 17), (1000003, 2, 61), (700001, 16, 15),
                                   (4200001, 8, 256)])
def test_against_a_stable_sort(t, k, e):
    import torch
    import moe_grouped_scaled_amd as M
    idx = _picks(t, k, e, t % 1000)
    need = M._native.LIB.mgs_moe_dispatch_workspace_bytes(t, k, e)
    ws = torch.full((need + 1024,), 0xA5, dtype=torch.uint8, device="cuda")
    print("case:", t, k, e, need, flush=True)
    row, splits = M.moe_dispatch(idx, e, workspace=ws[:need])
    torch.cuda.synchronize()
    assert bool((ws[need:] == 0xA5).all())
    flat = idx.view(-1).long()
    there = (flat >= 0) & (flat < e)
    key = torch.where(there, flat, e)
    order = torch.sort(key, stable=True).indices
    want = torch.empty_like(order)
    want[order] = torch.arange(order.numel(), device="cuda")
    assert torch.equal(row.view(-1).long(), torch.where(there, want, -1))
    assert torch.equal(splits, torch.bincount(key, minlength=e + 1)[:e])


@pytest.mark.gpu
def test_rows_and_weights_past_the_border():
    """The whole dispatch there: rows and weights follow, and the same bits again."""
    import torch
    import moe_grouped_scaled_amd as M
    t, k, e, h = 150001, 4, 40, 8
    idx = _picks(t, k, e, 1)
    x, w = torch.randn((t, h), device="cuda").to(torch.bfloat16), torch.rand((t, k), device="cuda")
    rows, rw = torch.full((t * k, h), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((t * k,), -1.0, device="cuda")
    row, splits = M.moe_dispatch(idx, e, x, rows, weights=w, row_weights=rw)
    live = row >= 0
    used = int(splits.sum())
    assert used == int(live.sum()) and 524288 < t * k
    at, tok = row[live].long(), live.nonzero()[:, 0]
    assert torch.equal(rows[at], x[tok]) and torch.equal(rw[at], w[live])
    assert bool((rows[used:] == 7.0).all()) and bool((rw[used:] == -1.0).all())
    again, _ = M.moe_dispatch(idx, e)
    assert torch.equal(again, row)


@pytest.mark.gpu
def test_time_grows_with_the_slots():
    """Eight times the slots: eight times the time where it is linear (64 times where every block reads all counts); twice
    that is allowed."""
    import torch
    import moe_grouped_scaled_amd as M

    def best(t):
        idx = _picks(t, 8, 256, 0)
        M.moe_dispatch(idx, 256)
        times = []
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            M.moe_dispatch(idx, 256)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    small, large = best(1 << 20), best(1 << 23)
    print("8.4 M slots %.3f ms, 67 M slots %.3f ms" % (small, large))
    assert large <= 16 * small
