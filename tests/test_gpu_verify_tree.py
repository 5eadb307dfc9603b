"""gdn_spec_verify_tree in batches that leave no SM idle (the persistent kernel) beside small ones (a unit's rows split
over a cluster): random trees at the widest group, refusals among good requests, checkpoint slots named twice."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from gated_deltanet_linear_conv1d_gb300 import synth  # noqa: E402
from oracle import oracle  # noqa: E402
from tests import attnref as R  # noqa: E402
from tests import gdnutil as U  # noqa: E402


@pytest.fixture(scope="module")
def b():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_deltanet_linear_conv1d_gb300 import build
    build.build()
    from gated_deltanet_linear_conv1d_gb300 import binding
    return binding


@pytest.fixture
def err():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def by_path(w, par, requests):
    """The oracle's result of every node of the given requests by its own path from a copy of the live slot."""
    P = par.shape[1]
    toks, lens, live = [], [], []
    for n in requests:
        for p in range(P):
            path, at = [], p
            while at >= 0:
                path.append(n * P + at)
                at = int(par[n, at])
            toks += path[::-1]
            lens.append(len(path))
            live.append(w["slot_idx"][n])
    r = oracle.forward(w["dims"], w["qkv0"][toks], w["conv_w"], np.ascontiguousarray(w["conv_hist"][live]),
                       np.ascontiguousarray(w["state"][live]), synth.pack_offsets(np.array(lens)),
                       np.arange(len(lens), dtype=np.int32), w["alpha"][toks], w["beta"][toks], w["z"][toks], w["gamma"],
                       w["eps"], inplace=True)
    last = np.cumsum(lens) - 1
    return r["o"][last], r["ogate"][last], r["state"], r["conv_hist"]


def verify(b, w, par, err=None):
    """(device workload after the call, o, ogate), both outputs filled with 7 before."""
    g, (N, P) = w["dims"], par.shape
    d = U.to_device(w)
    o = torch.full((N * P, g.num_v_heads, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    og = torch.full((N * P, g.num_v_heads * 128), 7.0, dtype=torch.bfloat16, device="cuda")
    b.gdn_spec_verify_tree(b.make_dims(g, w["num_slots"]), d["qkv0"], d["conv_w"], d["conv_hist"], d["state"],
                           d["slot_idx"], d["spec_slot_idx"], torch.from_numpy(par).cuda(), d["alpha"], d["beta"], d["z"],
                           d["gamma"], w["eps"], o=o, ogate=og, dev_err=err)
    return d, o, og


def check(w, par, requests, d, o, og):
    P = par.shape[1]
    ro, rg, state, hist = by_path(w, par, requests)
    rows = torch.tensor([n * P + p for n in requests for p in range(P)], device="cuda")
    U.check_out(U.host_f64_from_bf16(o[rows]), ro, "o")
    U.check_out(U.host_f64_from_bf16(og[rows]), rg, "ogate")
    ck = torch.from_numpy(w["spec_slot_idx"][requests].reshape(-1).astype(np.int64)).cuda()
    U.check_state(d["state"][ck].cpu().numpy(), state, U.STATE_REL_L2_DECODE, "checkpoints")
    np.testing.assert_array_equal(U.host_bits(d["conv_hist"][ck]), hist)


@pytest.mark.parametrize("geom,N,P", [(synth.Dims(2, 16, 128, 128, 4), 80, 8), (synth.Dims(4, 4, 128, 128, 4), 45, 8),
                                      (synth.FULL_HEADS, 10, 8)])
def test_random_trees_in_persistent_batches(b, err, geom, N, P):
    """More units than SMs; eight value heads a key head and eight nodes leave the ring two stages."""
    w = synth.spec_workload(geom, N, P, seed=P + N)
    par = R.tree(N, P, seed=N)[0].numpy()
    got = verify(b, w, par, err)
    assert b.gdn_read_device_error(err) == 0
    check(w, par, list(range(0, N, 7)), *got)
    again = verify(b, w, par, err)
    for x, y in zip((got[0]["state"], got[0]["conv_hist"], got[1], got[2]),
                    (again[0]["state"], again[0]["conv_hist"], again[1], again[2])):
        assert torch.equal(x, y)


@pytest.mark.parametrize("what,flag", [("parent", "TREE"), ("slot", "SLOT"), ("padding", None), ("all", "both")])
@pytest.mark.parametrize("N", [6, 64])
def test_refused_requests_among_good_ones(b, err, N, what, flag):
    """Bad parents, slots out of the pool and padding spread through a batch: those requests write nothing, the rest is
    as it should be. 64 requests at 4/12 heads are 256 units, of a kernel whose copies and consumers have to skip the
    same ones; 6 are split over clusters."""
    geom, P = synth.RANK_HEADS, 5
    w = synth.spec_workload(geom, N, P, seed=N)
    par = R.tree(N, P, seed=3)[0].numpy()
    clean = [w["slot_idx"].copy(), w["spec_slot_idx"].copy()]
    skipped = [n for n in range(N) if n % 3 == 1]
    for i, n in enumerate(skipped):
        kind = {"parent": 0, "slot": 2, "padding": 4}.get(what, 0) + (i % 2 if what != "all" else i % 6)
        if kind == 0:
            par[n, 3] = 3
        elif kind == 1:
            par[n, 0] = -2
        elif kind == 2:
            w["slot_idx"][n] = w["num_slots"]
        elif kind == 3:
            w["spec_slot_idx"][n, P - 1] = -1
        else:
            w["slot_idx"][n] = -1 if kind == 4 else -2 ** 31
    d, o, og = verify(b, w, par, err)
    want = {"TREE": b.GDN_DEVERR_TREE, "SLOT": b.GDN_DEVERR_SLOT, None: 0}.get(flag, b.GDN_DEVERR_TREE | b.GDN_DEVERR_SLOT)
    if what == "all" and len(skipped) < 3:
        want = b.GDN_DEVERR_TREE
    assert b.gdn_read_device_error(err) == want
    good = [n for n in range(N) if n not in skipped]
    check(w, par, good[::4], d, o, og)
    rows = torch.tensor([n * P + p for n in skipped for p in range(P)], device="cuda")
    assert bool((o[rows] == 7.0).all()) and bool((og[rows] == 7.0).all())
    still = torch.from_numpy(np.concatenate([clean[0], clean[1][skipped].reshape(-1)]).astype(np.int64)).cuda()
    host = still.cpu().numpy()
    assert torch.equal(d["state"][still].cpu(), torch.from_numpy(w["state"][host]))
    np.testing.assert_array_equal(U.host_bits(d["conv_hist"][still]), w["conv_hist"][host])


@pytest.mark.parametrize("N", [3, 50])
def test_a_checkpoint_slot_named_twice(b, err, N):
    """Nodes that nothing continues from may share a slot, the last one's state stays there. A node that continues from
    one whose slot an other node has taken since has lost its parent's state: the request is refused."""
    geom, P = synth.RANK_HEADS, 6
    w = synth.spec_workload(geom, N, P, seed=11)
    par = np.array([[-1, 0, 0, 1, 1, 2]] * N, np.int32)
    free = w["spec_slot_idx"].copy()
    w["spec_slot_idx"][:, 3] = w["spec_slot_idx"][:, 5]  # leaves 3 and 5 in one slot
    w["spec_slot_idx"][0, 4] = w["spec_slot_idx"][0, 2]  # in request 0 node 4 takes the slot of node 2, 5's parent
    chain = N - 1  # a chain never reads a state again, whatever slots it names
    par[chain] = np.arange(-1, P - 1)
    w["spec_slot_idx"][chain] = free[chain, 0]
    d, o, og = verify(b, w, par, err)
    assert b.gdn_read_device_error(err) == b.GDN_DEVERR_SLOT
    assert bool((o[:P] == 7.0).all()) and bool((og[:P] == 7.0).all())
    ck = free[0].astype(np.int64)
    assert torch.equal(d["state"][torch.from_numpy(ck).cuda()].cpu(), torch.from_numpy(w["state"][ck]))
    good = list(range(1, N, 7)) + [chain]
    ro, rg, state, hist = by_path(w, par, good)
    rows = torch.tensor([n * P + p for n in good for p in range(P)], device="cuda")
    U.check_out(U.host_f64_from_bf16(o[rows]), ro, "o")
    U.check_out(U.host_f64_from_bf16(og[rows]), rg, "ogate")
    for i, n in enumerate(good):
        for p in range(P):
            if p in ([P - 1] if n == chain else [0, 1, 2, 4, 5]):  # whose state stays
                s = int(w["spec_slot_idx"][n, p])
                U.check_state(d["state"][s].cpu().numpy(), state[i * P + p], U.STATE_REL_L2_DECODE, f"{n}, {p}")
                np.testing.assert_array_equal(U.host_bits(d["conv_hist"][s]), hist[i * P + p])
