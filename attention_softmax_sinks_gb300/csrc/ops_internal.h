// Internal interface of the kernels around attention, as abi.cu sees it: the
// standalone router, QKV bias + rotary + K/V write, the bias-seeded linear
// layer, and the expert layer behind the router (each kernel file includes only
// the headers it needs).
#pragma once
#include "experts_args.h"
#include "grouped_args.h"
#include "linear_args.h"
#include "lora_args.h"
#include "rope_args.h"
#include "router_args.h"
#include "router_scores_args.h"
#include "shared_args.h"
