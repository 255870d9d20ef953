// What the attention kernels share: the call's arguments and launchers.
#pragma once

#include "kvcache.cuh"
