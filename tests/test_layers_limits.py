"""The largest sizes that linear attention and group norm take, and what is refused above them.  CPU only: the size
queries and the argument checks run on the host before anything is enqueued."""
import pytest
import torch

from newton_solve_nonlinear_b200 import binding
from tests.test_layers_refusals import L, _norm  # noqa: F401 (L is a fixture)

INT_MAX = 2 ** 31 - 1


@pytest.mark.parametrize("C", [1, 5, 8])
@pytest.mark.parametrize("N,S", [(1, INT_MAX), (1, INT_MAX - 100), (1, 2 ** 31 - 3_000_000), (3, INT_MAX // 3)])
def test_norm_workspace_of_the_longest_sequences(L, N, S, C):  # noqa: F811
    """Rows are dealt to a fixed number of CTAs, so the workspace does not grow with S from some length on."""
    for size in (L.pararnn_group_norm_workspace_size, L.pararnn_group_norm_backward_workspace_size):
        shape = lambda s: _norm(N=N, S=s, C=C, groups=1)
        base = size(shape(2 ** 29 // N))
        assert base > 256
        assert base // 2 <= size(shape(S)) <= 2 * base


@pytest.mark.parametrize("C,groups", [(8, 1), (7, 7), (64, 4)])
@pytest.mark.parametrize("N", [INT_MAX, INT_MAX - 1, INT_MAX - 200])
def test_norm_of_the_most_rows_fills_the_card(L, N, C, groups):  # noqa: F811
    """One row per statistic: the backward pass keeps a row of partial sums for each CTA, as many as for fewer rows."""
    size = lambda n: L.pararnn_group_norm_backward_workspace_size(_norm(N=n, S=1, C=C, groups=groups))
    assert size(N) == size(2 ** 24) >= 148 * 2 * C * 4


@pytest.mark.parametrize("S,groups", [(1, 1), (2, 1), (1, 64)])
def test_norm_channels(L, S, groups):  # noqa: F811
    """Channels are counted in 32 bits, in two sums a channel and in strides that may pass the end: up to 2^30."""
    for size in (L.pararnn_group_norm_workspace_size, L.pararnn_group_norm_backward_workspace_size):
        query = lambda C: size(_norm(N=1, S=S, C=C, groups=groups))
        assert query(2 ** 30) >= 256
        for C in (2 ** 30 + groups, INT_MAX // groups * groups):
            assert query(C) == 0


FAR = 2 ** 32 + 3  # what a 32-bit count would take for 3


def _far(*shape):
    return torch.zeros(*(1 for _ in shape)).expand(*shape)  # no memory behind it


@pytest.mark.parametrize("shape", [(FAR, 1, 1, 1), (1, FAR, 1, 1), (1, 1, FAR, 1)])
def test_attention_sizes_beyond_32_bits_are_refused(shape):
    q = _far(*shape)
    ld = _far(shape[2])
    with pytest.raises(ValueError, match="below 2\\*\\*31"):
        binding.linear_attention(q, q, q, ld)
    with pytest.raises(ValueError, match="below 2\\*\\*31"):
        binding.linear_attention_backward(q, q, q, ld, q)


@pytest.mark.parametrize("rows,slots", [(FAR, FAR), (3, FAR)])
def test_step_sizes_beyond_32_bits_are_refused(rows, slots):
    q, state = _far(rows, 1, 1), _far(slots, 1, 1, 1)
    with pytest.raises(ValueError, match="below 2\\*\\*31"):
        binding.linear_attention_step(q, q, q, _far(1), state, slots=torch.zeros(3, dtype=torch.int32))


@pytest.mark.parametrize("shape", [(FAR, 1), (1, FAR), (1, FAR, 1), (3, 2 ** 16, 2 ** 16, 1), (1, 3, FAR)])
def test_norm_sizes_beyond_32_bits_are_refused(shape):
    x = _far(*shape)
    with pytest.raises(ValueError, match="below 2\\*\\*31"):
        binding.group_norm(x, 1)
    with pytest.raises(ValueError, match="below 2\\*\\*31"):
        binding.group_norm_backward(x, _far(shape[0], 1, 2), x, 1)


class _Elsewhere:
    """What the binding looks at of a stream or a buffer, on a second device."""
    device, cuda_stream, is_cuda = torch.device("cuda", 1), 0, True

    def get_device(self):
        return 1

    def data_ptr(self):
        return 1 << 40

    def numel(self):
        return 1 << 20

    def is_contiguous(self):
        return True


def test_streams_of_another_device_are_refused(monkeypatch):
    """Such a call ran on the current stream of its tensors' device instead, without the order that was asked for."""
    monkeypatch.setattr(torch.cuda, "stream", lambda s: pytest.fail("entered the stream"))
    z = torch.zeros
    q = z(1, 2, 4, 8)
    other = dict(stream=_Elsewhere())
    for call in (lambda: binding.linear_attention(q, q, q, z(4), **other),
                 lambda: binding.linear_attention_backward(q, q, q, z(4), q, **other),
                 lambda: binding.linear_attention_step(q[:, 0], q[:, 0], q[:, 0], z(4), z(1, 4, 8, 8), **other),
                 lambda: binding.group_norm(z(3, 4), 1, **other),
                 lambda: binding.group_norm_backward(z(3, 4), z(3, 1, 2), z(3, 4), 1, **other)):
        with pytest.raises(ValueError, match="stream"):
            call()


def test_workspaces_of_another_device_are_refused():
    with pytest.raises(ValueError, match="workspace"):
        binding._workspace(1024, "pararnn_group_norm", _Elsewhere(), torch.device("cuda", 0))
    assert binding._workspace(1024, "pararnn_group_norm", _Elsewhere(), torch.device("cuda", 1))[1:] == (1 << 40, 1 << 20)


@pytest.mark.parametrize("which", range(4))
def test_attention_refuses_to_drop_a_gradient(which):
    """The calls record no graph; the gradients come from the backward call.  Under no_grad the operands may be leaves."""
    z = torch.zeros
    q, k, v, s0 = a = (z(1, 2, 4, 8), z(1, 2, 4, 8), z(1, 2, 4, 8), z(1, 4, 8, 8))
    a[which].requires_grad_()
    calls = [lambda: binding.linear_attention(q, k, v, z(4), s0=s0),
             lambda: binding.linear_attention_step(q[:, 0], k[:, 0], v[:, 0], z(4), s0)]
    for call in calls:
        with pytest.raises(ValueError, match="no graph"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="CUDA"):  # the backward call takes the same leaves
        binding.linear_attention_backward(q, k, v, z(4), q, s0=s0)


@pytest.mark.parametrize("which", range(4))
def test_norm_refuses_to_drop_a_gradient(which):
    x, w, b, gate = a = (torch.zeros(3, 4), torch.zeros(4), torch.zeros(4), torch.zeros(3, 4))
    a[which].requires_grad_()
    with pytest.raises(ValueError, match="no graph"):
        binding.group_norm(x, 1, w, b, gate=gate)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
        binding.group_norm(x, 1, w, b, gate=gate)
    with pytest.raises(ValueError, match="CUDA"):
        binding.group_norm_backward(x, torch.zeros(3, 1, 2), torch.zeros(3, 4), 1, w, b, gate=gate)


def test_decays_that_are_leaves_serve_under_no_grad():
    """No gradient is lost there; the backward call, which has none for the decays, refuses them always."""
    z = torch.zeros
    q, ld = z(1, 2, 4, 8), z(4).requires_grad_()
    with torch.no_grad():
        for call in (lambda: binding.linear_attention(q, q, q, ld),
                     lambda: binding.linear_attention_step(q[:, 0], q[:, 0], q[:, 0], ld, z(1, 4, 8, 8))):
            with pytest.raises(ValueError, match="CUDA"):
                call()
        with pytest.raises(ValueError, match="gradient"):
            binding.linear_attention_backward(q, q, q, ld, q)
    with pytest.raises(ValueError, match="gradient"):
        binding.linear_attention_step(q[:, 0], q[:, 0], q[:, 0], ld, z(1, 4, 8, 8))
