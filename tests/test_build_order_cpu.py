"""The contract library, the probes and the oracle are built and loaded before anything that
needs a C++ compiler with torch's headers, so that a policy head that cannot be built takes
nothing else with it, and says so."""

import pytest

import __graft_entry__ as entry
from bitwise_consistent_linear_amd import api, build
from oracle import oracle


def test_a_failing_binding_leaves_the_rest_built(monkeypatch):
    done = []

    def fail(*a, **k):
        raise RuntimeError("failed to build _policy_binding.so")

    def step(name):
        return lambda *a, **k: done.append(name)

    monkeypatch.setattr(build, "build", step("contract"))
    monkeypatch.setattr(build, "build_probe", step("probe"))
    monkeypatch.setattr(oracle, "build", step("oracle"))
    monkeypatch.setattr(api, "lib", step("contract loaded"))
    monkeypatch.setattr(build, "_build", step("policy"))
    monkeypatch.setattr(build, "build_policy_binding", fail)
    monkeypatch.setattr(api, "_policy", step("policy loaded"))
    with pytest.raises(RuntimeError, match="_policy_binding"):
        entry.build()
    assert done == ["contract", "probe", "oracle", "contract loaded", "policy"]
