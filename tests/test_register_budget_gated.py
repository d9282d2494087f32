"""Host check (no GPU): the gated decode's combine keeps the register budget of the
other combines (test_register_budget.py): a CTA of it fits on an SM beside a CTA of
the next launch's main kernel."""
from test_register_budget import SM_REGISTERS, _alloc, _pick, registers   # noqa: F401 (a fixture)


def test_gated_combine_fits_beside_the_next_main_cta(registers):   # noqa: F811
    main = {**_pick(registers, r"gemv_lut8_kernelILi\dELb\dELb0E"), **_pick(registers, r"gemv_lut8_multi_kernel")}
    worst_main = max(_alloc(n) for n in main.values())
    combine = _pick(registers, r"gemv_combine_gated_kernel")
    assert len(combine) == 2
    for name, n in combine.items():
        total = 512 * worst_main + 256 * _alloc(n)
        assert total <= SM_REGISTERS, f"{name}: {n} registers; with a {worst_main}-register main CTA: {total}"
