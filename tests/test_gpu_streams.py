"""Calls on another stream than the current one: what they allocate for
themselves belongs to the stream that uses it.

A stalled stream is given work; memory that the call has freed by then must
not reach the current stream's tensors, which are filled at once and have to
stay as they are when the stalled work runs."""
import pytest
import torch

import exact_lloyd_means_amd as fk

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"


def stall(stream):
    """Some tens of milliseconds of work."""
    with torch.cuda.stream(stream):
        a = torch.ones(4096, 4096, device="cuda")
        for _ in range(30):
            a = (a @ a) * 2.0 ** -12
    return a


class Bystanders:
    """Tensors of these sizes in bytes made on the current stream now."""

    def __init__(self, sizes):
        self.t = [torch.full((n,), 0x5a, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(8)]

    def untouched(self):
        torch.cuda.synchronize()
        return all(bool((t == 0x5a).all()) for t in self.t)


def points(B=2, N=20000, K=64, d=32):
    g = torch.Generator("cuda").manual_seed(0)
    X = torch.randn(B, N, d, device="cuda", generator=g)
    return X, X[:, :K].clone(), torch.randint(0, K, (B, N), device="cuda", generator=g, dtype=torch.int32)


@pytest.mark.parametrize("handle", [False, True])     # a stream object, and its address
@pytest.mark.parametrize("what", ["assign", "sort", "update", "update_bias", "lloyd", "kmeans"])
def test_workspaces_of_a_side_stream(what, handle):
    side = torch.cuda.Stream()
    X, C, labels = points()
    (B, N, d), K = X.shape, C.shape[1]
    f32, i32 = dict(device="cuda"), dict(dtype=torch.int32, device="cuda")
    out = dict(labels=torch.empty(B, N, **i32), counts=torch.empty(B, K, **i32), offsets=torch.empty(B, K + 1, **i32),
               order=torch.empty(B, N, **i32), C=torch.empty(B, K, d, **f32), bias=torch.empty(B, K, **f32))

    def call(stream, o):
        if what == "assign":
            fk.fk_assign(X, C, o["labels"], stream=stream)
        elif what == "sort":
            fk.fk_sort_labels(labels, K, o["counts"], o["offsets"], o["order"], stream=stream)
        elif what == "update":
            fk.fk_update(X, labels, C, o["C"], None, o["counts"], stream=stream, deterministic=True)
        elif what == "update_bias":
            fk.fk_update_bias(X, labels, C, o["C"], None, o["counts"], o["bias"], stream=stream, deterministic=True)
        elif what == "lloyd":
            fk.fk_lloyd(X, o["C"], o["labels"], o["counts"], 3, stream=stream, deterministic=True)
        else:
            o["labels"], o["C"], _ = fk.batch_kmeans_euclid(X, K, 3, init="first", stream=stream, deterministic=True)
        return o
    want, got = ({k: torch.zeros_like(v) for k, v in out.items()} for _ in range(2))
    for o in (want, got):
        o["C"].copy_(C)                                # fk_lloyd starts from it
    call(None, want)
    ws = fk.workspace_size(fk.problem(B, N, K, d, torch.float32, True))
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    stall(side)
    call(side.cuda_stream if handle else side, got)
    by = Bystanders([ws, fk.workspace_size(fk.problem(B, N, K, d, torch.float32)), 4 * B * N, 4 * B * K])
    assert by.untouched()
    for k in want:
        assert torch.equal(got[k], want[k]), k


def test_kmeans_prepares_its_points_on_the_stream():
    # strided points and a tensor of centroids are copied first; the current stream is the stalled one
    side = torch.cuda.Stream()
    X, C, _ = points()
    X = X.transpose(1, 2).contiguous().transpose(1, 2)
    want = fk.batch_kmeans_euclid(X, 64, 3, init=C, deterministic=True)
    torch.cuda.synchronize()
    keep = stall(torch.cuda.current_stream())
    got = fk.batch_kmeans_euclid(X, 64, 3, init=C, deterministic=True, stream=side)
    side.synchronize()
    with torch.cuda.stream(side):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    torch.cuda.synchronize()
    del keep


def test_the_default_streams_address():
    X, C, _ = points()
    a, b = (torch.empty(X.shape[:2], dtype=torch.int32, device="cuda") for _ in range(2))
    torch.cuda.synchronize()
    fk.fk_assign(X, C, a)
    with torch.cuda.stream(torch.cuda.Stream()):
        fk.fk_assign(X, C, b, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
