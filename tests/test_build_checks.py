"""The build's check of the compiler's resource remarks."""
from embedding_table_gather_amd.build import spilled

REMARKS = """a.hip:1:1: remark: Function Name: first [-Rpass-analysis=kernel-resource-usage]
a.hip:1:1: remark:     SGPRs Spill: 154 [-Rpass-analysis=kernel-resource-usage]
a.hip:1:1: remark:     VGPRs Spill: {} [-Rpass-analysis=kernel-resource-usage]
a.hip:2:1: remark: Function Name: second [-Rpass-analysis=kernel-resource-usage]
a.hip:2:1: remark:     VGPRs Spill: {} [-Rpass-analysis=kernel-resource-usage]
"""


def test_spilled_vector_registers_are_named():
    assert spilled(REMARKS.format(0, 0)) == [] and spilled("") == []
    assert spilled(REMARKS.format(0, 26)) == ["second: 26"]
    assert spilled(REMARKS.format(4, 1)) == ["first: 4", "second: 1"]
