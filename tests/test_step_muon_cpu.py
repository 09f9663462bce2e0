"""RankStep with Muon: its choices and refusals (no call reaches the device)."""
import pytest
import torch

CPU = torch.device("cpu")


@pytest.fixture(scope="module")
def zm():
    import zero_partitioned_mixed_partition_amd as m
    return m


@pytest.fixture(scope="module")
def st():
    from zero_partitioned_mixed_partition_amd import step as s
    return s


def _make(zm, st, numels, shapes, ranks=1, rank=0, **kw):
    plan = zm.zero_partition_plan(numels, ranks, 1)
    kw = dict(dict(per_param=True, muon=st.MuonHyper()), **kw)
    return st.RankStep(plan, rank, 1, st.Hyper(), 0.0, CPU, muon_shapes=shapes, **kw)


def test_state_of_matrices_and_of_the_rest(zm, st):
    rs = _make(zm, st, [12, 5, 20, 6], {0: (3, 4), 2: (4, 5)})
    assert rs.muon_segments == {0: (3, 4), 2: (4, 5)}
    assert [x.numel() for x in rs.master_tensors] == [12, 5, 20, 6] == [x.numel() for x in rs.exp_avg_tensors]
    assert [x.numel() for x in rs.exp_avg_sq_tensors] == [0, 5, 0, 6]
    plain = st.RankStep(zm.zero_partition_plan([12, 5], 1, 1), 0, 1, st.Hyper(), 0.0, CPU, per_param=True)
    assert plain.muon_segments == {} and [x.numel() for x in plain.exp_avg_sq_tensors] == [12, 5]


def test_a_matrix_of_another_rank_is_not_this_ranks(zm, st):
    """Two ranks of 12 elements: rank 0 holds the matrix whole, rank 1 nothing of it."""
    assert _make(zm, st, [12, 12], {0: (3, 4)}, 2, 0).muon_segments == {0: (3, 4)}
    assert _make(zm, st, [12, 12], {0: (3, 4)}, 2, 1).muon_segments == {}


def test_refusals(zm, st):
    with pytest.raises(ValueError, match="whole matrix on one rank"):
        _make(zm, st, [20, 4], {0: (4, 5)}, 2, 0)
    with pytest.raises(ValueError, match="no 3 x 5 matrix"):
        _make(zm, st, [12], {0: (3, 5)})
    with pytest.raises(ValueError, match="no -3 x -4 matrix"):
        _make(zm, st, [12], {0: (-3, -4)})
    with pytest.raises(ValueError, match="names tensor 1"):
        _make(zm, st, [12], {1: (3, 4)})
    with pytest.raises(ValueError, match="per-parameter state"):
        _make(zm, st, [12], {0: (3, 4)}, per_param=False)
    with pytest.raises(ValueError, match="state_bits is 32"):
        _make(zm, st, [12], {0: (3, 4)}, state_bits=8)
    with pytest.raises(ValueError, match="without Muon's settings"):
        _make(zm, st, [12], {0: (3, 4)}, muon=None)
