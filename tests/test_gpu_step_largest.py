"""The largest counts that the operators of a step of samples take."""
import pytest
import torch

import samples_util as S

pytestmark = pytest.mark.gpu


def test_room_for_the_most_tokens():
    """total_q = 2^31 - 1: all that no request has is -1, up to the last."""
    import block_sparse_top_msa_gb300 as msa
    if torch.cuda.mem_get_info()[0] < 48 << 30:
        pytest.skip("48 GB wanted")
    n, most = 16384, 2**31 - 1
    table = torch.arange(n, dtype=torch.int32, device="cuda")[:, None].contiguous()
    ones = torch.ones(n, dtype=torch.int32, device="cuda")
    t = msa.msa_step_tables(table, 5 * ones, torch.arange(n, dtype=torch.int32, device="cuda"), ones, total_q=most, num_pages=n)
    assert msa.msa_read_device_fault() == 0
    assert t.cu_seqlens_q.tolist() == list(range(n + 1))
    assert torch.equal(t.slots[:n], torch.arange(n, device="cuda") * 128 + 4) and bool((t.positions[:n] == 4).all())
    for x in (t.token_rows, t.positions, t.slots):
        assert all(bool((x[lo : lo + 2**28] == -1).all()) for lo in range(n, most, 2**28))


def test_rows_of_the_most_pages_in_one_table():
    """A table of 2^28 places a row, of which a request holds three."""
    import block_sparse_top_msa_gb300 as msa
    width = 2**28 + 3
    table = torch.full((2, width), -1, dtype=torch.int32, device="cuda")
    table[:, :3] = torch.tensor([[4, 5, 6], [4, 5, 7]], dtype=torch.int32)
    t = msa.msa_step_tables(table, S.ints([384, 300]), S.ints([0, 1]), S.ints([1, 1]), total_q=2, num_pages=8)
    assert torch.equal(t.page_table[:, :4].cpu(), torch.tensor([[4, 5, 6, -1], [4, 5, 7, -1]], dtype=torch.int32))
    assert bool((t.page_table[:, 3:] == -1).all()) and t.group_blocks.tolist() == [2, 0] and t.slots.tolist() == [6 * 128 + 127, 7 * 128 + 43]
    assert msa.msa_read_device_fault() == 0


def test_a_path_with_much_more_room_than_nodes():
    import block_sparse_top_msa_gb300 as msa
    n = 2**24 + 5
    path, length, after = msa.msa_draft_path(S.ints([7, 8, 9]), S.ints([0, 7, 5]), S.mask_rows([-1, 0, 1]).cuda(), S.ints([0, 3]), max_path=n)
    assert path[0, :2].tolist() == [0, 1] and bool((path[0, 2:] == -1).all()) and length.tolist() == [2] and after.tolist() == [8]
    assert msa.msa_read_device_fault() == 0
