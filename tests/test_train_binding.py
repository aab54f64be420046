"""What the binding of the embedding and the losses does before a call (CPU only)."""
import pytest


@pytest.fixture(scope="module")
def lp():
    import lm_head_linear_tcgen05_gb300 as mod
    return mod


def _ranges(ref):
    part = ref._obj
    return [(part.shards[k].vocab_start, part.shards[k].vocab_end) for k in range(part.n_shards)]


def test_a_partition_that_changes_is_read_again(lp):
    """Any object with the three fields is a partition; one of an ordinary class hashes by identity, so what
    was read from it before says nothing of what it holds now."""
    class Partition:
        vocab_real, vocab_padded, ranges = 1000, 1024, ((0, 1024),)

    part = Partition()
    assert _ranges(lp._partition_ref(part)) == [(0, 1024)]
    part.ranges = ((0, 100), (100, 512), (512, 1024))
    assert _ranges(lp._partition_ref(part)) == [(0, 100), (100, 512), (512, 1024)]
    part.vocab_real, part.local = 600, True
    assert (lp._partition_ref(part)._obj.vocab_real, lp._partition_ref(part)._obj.local) == (600, 1)

    class Derived(lp.VocabPartition):
        __hash__ = object.__hash__

        def __eq__(self, other):
            return self is other

    part = Derived(1000, 1024, ((0, 1024),))
    assert _ranges(lp._partition_ref(part)) == [(0, 1024)]
    object.__setattr__(part, "ranges", ((0, 24), (24, 1024)))
    assert _ranges(lp._partition_ref(part)) == [(0, 24), (24, 1024)]


def test_partitions_are_told_apart_by_value(lp):
    whole, halves = lp.VocabPartition(1000, 1024, ((0, 1024),)), lp.VocabPartition(1000, 1024, ((0, 512), (512, 1024)))
    local = lp.VocabPartition(1000, 1024, ((0, 1024),), local=True)
    listed = lp.VocabPartition(1000, 1024, [(0, 8), (8, 1024)])        # not hashable
    for _ in range(2):
        assert _ranges(lp._partition_ref(whole)) == [(0, 1024)] and lp._partition_ref(whole)._obj.local == 0
        assert _ranges(lp._partition_ref(halves)) == [(0, 512), (512, 1024)]
        assert lp._partition_ref(local)._obj.local == 1
        assert _ranges(lp._partition_ref(listed)) == [(0, 8), (8, 1024)]
        listed.ranges[:] = [(0, 16), (16, 1024)]
        assert _ranges(lp._partition_ref(listed)) == [(0, 16), (16, 1024)]
        listed.ranges[:] = [(0, 8), (8, 1024)]


@pytest.mark.parametrize("name,value", [("upstream", None), ("upstream", 2.0), ("grads", True), ("grads", False),
                                        ("metrics", True), ("metrics", False)])
def test_the_autograd_losses_refuse_what_autograd_gives(lp, name, value):
    """At the call, by name: not in the backward, after a forward that took the option."""
    import torch
    from lm_head_linear_tcgen05_gb300.autograd import policy_loss, preference_loss
    x, cu = torch.zeros(4, requires_grad=True), torch.tensor([0, 2, 4], dtype=torch.int32)
    with pytest.raises(TypeError, match=f"{name} is not an option"):
        policy_loss(x, x.detach(), x.detach(), **{name: value})
    with pytest.raises(TypeError, match=f"{name} is not an option"):
        preference_loss(x, cu, **{name: value})


def _outputs(lp, metrics=True):
    import torch
    return lp.LossOutputs(metrics=torch.arange(5, 11, dtype=torch.float32) if metrics else None, counts=None,
                          grad_logp=torch.zeros(3))


def test_the_loss_is_there_however_it_is_asked_for(lp):
    """Each question put to outputs of its own, so that none finds what an earlier one left."""
    import copy
    import pickle
    names = {"loss", "metrics", "counts", "grad_logp"}
    assert float(_outputs(lp)["loss"]) == 5.0 and float(_outputs(lp).get("loss")) == 5.0
    assert "loss" in _outputs(lp) and len(_outputs(lp)) == 4
    assert set(_outputs(lp)) == set(_outputs(lp).keys()) == set(reversed(_outputs(lp))) == names
    assert float(dict(_outputs(lp).items())["loss"]) == 5.0 and len(_outputs(lp).values()) == 4
    (lambda loss, metrics, counts, grad_logp: None)(**_outputs(lp))
    filled = {}
    filled.update(_outputs(lp))
    whole = (dict(_outputs(lp)), {**_outputs(lp)}, filled, _outputs(lp).copy(), copy.copy(_outputs(lp)),
             pickle.loads(pickle.dumps(_outputs(lp))), _outputs(lp) | {}, {} | _outputs(lp))
    assert all(set(w) == names and float(w["loss"]) == 5.0 for w in whole)
    assert float(_outputs(lp).pop("loss")) == 5.0 and float(_outputs(lp).setdefault("loss", 1.0)) == 5.0
    assert "loss" in repr(_outputs(lp))
    out = _outputs(lp)
    assert out["loss"] is out["loss"] and out["loss"].data_ptr() == out["metrics"].data_ptr()
    for take in (lambda o: o.pop("loss"), lambda o: o.__delitem__("loss")):
        out = _outputs(lp)
        take(out)
        assert "loss" not in out and out.get("loss") is None and len(out) == 3
    out = _outputs(lp)
    out["loss"] = 2.0
    assert out["loss"] == out.get("loss") == dict(out)["loss"] == 2.0
    # without metrics there is no loss
    none = _outputs(lp, metrics=False)
    assert "loss" not in none and none.get("loss") is None and set(none) == names - {"loss"}
    with pytest.raises(KeyError):
        none["loss"]
    with pytest.raises(KeyError):
        _outputs(lp)["grad"]


def test_an_embedding_without_shards_is_refused_alike(lp):
    """Under autograd with the library call's error."""
    import torch
    from lm_head_linear_tcgen05_gb300.autograd import embedding
    ids, part = torch.zeros(3, dtype=torch.int32), lp.VocabPartition(8, 8, ((0, 8),))
    for W in ([None], [torch.zeros(8, 8).tolist()], []):
        with pytest.raises((TypeError, ValueError)):
            lp.lp_embedding(ids, W, part)
        with pytest.raises((TypeError, ValueError)):
            embedding(ids, W, part)
